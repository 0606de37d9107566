// What the products' C entries share: how an operand is read, the tile and the
// split of a product, and its launches.
#pragma once

#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "gemm_launch.hpp"
#include "host_common.hpp"
#include "rows_kernel.hpp"

namespace dense {
namespace {

constexpr int64_t kWsAlign = 256;
// Byte limits of a tile's 31-bit load offsets: 256 rows of a rows-form
// operand, 64 inner rows of a columns-form one.
constexpr int64_t kMaxRowBytes = ((int64_t)1 << 31) / 256 - 64;
constexpr int64_t kMaxColBytes = ((int64_t)1 << 31) / 64 - 64;

// One operand of a product as the kernel reads it.
struct Operand {
    const void *src = nullptr;
    int64_t rs = 0, cs = 0;  // source strides in elements: along the dim and the inner dim
    int64_t dim = 0, inner = 0;
    int es = 2;
    bool cols = false;       // columns form
    bool packed = false;     // copied into the workspace first
    int64_t ld = 0;          // bytes between rows (inner rows for the columns form) as read
    int64_t pack_bytes = 0;
};

// Decides how an operand [dim, inner] is read: in place in rows form (inner
// contiguous) or, where the kernel has that form, columns form (dim
// contiguous), if 16-byte chunks are aligned, do not straddle a row's end and are
// within a tile's reach; otherwise from a packed copy.  Columns form has its inner rows one after the
// other, none repeated or overlapping: the kernel tells those past the end by
// the byte range that ends with the last one.
void plan_operand(Operand *o, bool allow_rows, bool allow_cols)
{
    const bool rows_ok = allow_rows && (o->cs == 1 || o->inner <= 1);
    const bool cols_ok = allow_cols && (o->rs == 1 || o->dim <= 1);
    const bool aligned = ((uintptr_t)o->src & 15) == 0;
    o->cols = cols_ok && !rows_ok;
    if (!rows_ok && !cols_ok)
        o->cols = !allow_rows;
    const int64_t len = o->cols ? o->dim : o->inner;     // contiguous length
    const int64_t pitch = (o->cols ? o->cs : o->rs) * o->es;
    const int64_t n = o->cols ? o->inner : o->dim;
    o->packed = !((rows_ok || cols_ok) && aligned && len * o->es % 16 == 0 &&
                  (n <= 1 || (pitch % 16 == 0 && (!o->cols || pitch >= len * o->es) &&
                              pitch <= (o->cols ? kMaxColBytes : kMaxRowBytes))));
    if (o->packed) {
        o->ld = round_up(len * o->es, 16);
        o->pack_bytes = round_up(o->ld * n, kWsAlign);
    } else {
        o->ld = n <= 1 ? round_up(len * o->es, 16) : pitch;
    }
}

// Workgroups of so many threads that copy an operand.
int64_t pack_wgs(const Operand &o, int threads = 256)
{
    return o.packed ? ceil_div((o.cols ? o.inner : o.dim) * (o.ld / 16), threads) : 0;
}

conv_i8_status_t check_reach(const Operand &o)
{
    if (o.ld > (o.cols ? kMaxColBytes : kMaxRowBytes) || !launch_fits(pack_wgs(o), 256))
        return CONV_I8_ERR_UNSUPPORTED;
    return CONV_I8_OK;
}

PackJob pack_job(const Operand &o, void *dst)
{
    PackJob j;
    memset(&j, 0, sizeof j);
    if (!o.packed)
        return j;
    j.src = o.src;
    j.dst = dst;
    j.rows = o.cols ? o.inner : o.dim;
    j.cols = o.cols ? o.dim : o.inner;
    j.rs = o.cols ? o.cs : o.rs;
    j.cs = o.cols ? o.rs : o.cs;
    j.chunks = o.ld / 16;
    j.items = j.rows * j.chunks;
    return j;
}

// Both jobs of a launch; returns its workgroups.
int64_t pack_jobs(const Operand &a, void *da, const Operand &b, void *db, PackArgs *p, int threads = 256)
{
    p->job[0] = pack_job(a, da);
    p->job[1] = pack_job(b, db);
    p->first = (int)pack_wgs(a, threads);
    return pack_wgs(a, threads) + pack_wgs(b, threads);
}

bool launch_pack(const Operand &a, void *da, const Operand &b, void *db, hipStream_t stream)
{
    PackArgs p;
    const int64_t wgs = pack_jobs(a, da, b, db, &p);
    if (wgs == 0)
        return true;
    const dim3 grid((unsigned)wgs), block(256);
    if (a.es == 1)
        hipLaunchKernelGGL(pack_kernel<uint8_t>, grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL(pack_kernel<uint16_t>, grid, block, 0, stream, p);
    return hipGetLastError() == hipSuccess;
}

// Tile and split of one product.
struct GemmPlan {
    int tile = 0, splits = 1;
    int tiles_m = 0, tiles_n = 0, nstages = 0, kchunk = 0;
    int terms = 1;  // of the first operand, each a product of its own
    int part_ld = 0;
    int64_t part_bytes = 0;
    bool joined() const { return splits > 1 || terms > 1; }
};

// Microseconds a product takes with a tile and a split: the stages of the CU
// that has the most workgroups, what a round of workgroups costs besides
// (filling the pipeline, the epilogue; workgroups that share a CU hide it from
// each other), the output's bytes, and for a split the second launch and the
// pass over the partial sums.  The constants are a fit to measured times.  Of 27
// shapes from 64x1024x1024 to 8192x8192x2048, all tiles and splits timed, its
// choice is within 8 % of the best one for 24; 528x1072x5312, 1024x2048x4096 and
// 64x8192x8192 take 13 to 17 % more.
struct TileCost {
    double stage;  // us per 64 bytes of the inner dimension of one workgroup
    double alone;  // the same of the only one on its CU
    double round;  // us per round of workgroups
    double out;    // us per 10^6 outputs
};
constexpr TileCost kCost[kTiles] = {
    {0.536, 0.536, 8.2, 0.45},
    {0.259, 0.259, 4.4, 0.45},
    {0.089, 0.089, 3.8, 0.90},
    {0.194, 0.194, 4.8, 0.45},
};
// Of 8-bit floating point, whose stage has twice the products of a 16-bit one and waits for
// its scales.  Of 22 shapes from 64x1024x1024 to 8192x8192x2048 its choice is within 4 % of the
// best one for all (128x512x4096: 10.1 us in four parts, 14.7 unsplit as the constants above would
// have it); of 17 to 100 rows with 8192 to 32768 rows of w it is 2 to 24 % from it.
constexpr TileCost kCostF8[kTiles] = {
    {0.550, 0.550, 8.2, 0.45},
    {0.275, 0.275, 4.4, 0.45},
    {0.120, 0.155, 3.8, 0.90},
    {0.290, 0.290, 4.8, 0.45},
};

double gemm_cost(const TileCost *costs, int tile, int64_t M, int64_t N, int64_t kbytes, int splits)
{
    const Tile &t = kTile[tile];
    const TileCost &c = costs[tile];
    const int64_t wgs = ceil_div(M, t.tm) * ceil_div(N, t.tn) * splits;
    const int64_t per_cu = ceil_div(wgs, kCUs);
    const double stages = (double)(per_cu * ceil_div(kbytes, 64 * splits)) * (per_cu > 1 ? c.stage : c.alone);
    const double rounds = (double)ceil_div(per_cu, t.occ) * c.round;
    const double busy = t.occ == 1 ? stages + rounds : stages + c.round > rounds ? stages + c.round : rounds;
    const double mn = 1.0e-6 * (double)M * (double)N;
    return busy + (splits > 1 ? 4.4 + 1.2 * mn * splits : c.out * mn);
}

// The same of both gradients' products in one launch with tile kPairTile:
// either all CUs work through both, or the longer reduction lasts longest.
double pair_cost(int64_t M, int64_t N, int64_t K, int es = 2, const TileCost *costs = kCost)
{
    const Tile &t = kTile[kPairTile];
    const TileCost &c = costs[kPairTile];
    const double sx = (double)ceil_div(es * N, 64), sw = (double)ceil_div(es * M, 64);
    const double all = (sx * (double)ceil_div(M, t.tm) + sw * (double)ceil_div(N, t.tm)) * (double)ceil_div(K, t.tn) / kCUs;
    const double longest = sx > sw ? sx : sw;
    return (all > longest ? all : longest) * c.alone + c.round + c.out * 1.0e-6 * (double)(M + N) * (double)K;
}

// CONV_I8_DENSE_TILE, for tests and sweeps: "128x128" names a tile for every
// product, "128x128/4" a tile and a split.
struct Forced {
    bool on = false;
    int tile = 0, split = 0;  // split 0: the plan's choice
};

conv_i8_status_t forced_tile(Forced *f)
{
    const char *s = getenv("CONV_I8_DENSE_TILE");
    if (!s || !*s)
        return CONV_I8_OK;
    const char *slash = strchr(s, '/');
    const size_t len = slash ? (size_t)(slash - s) : strlen(s);
    while (f->tile < kTiles && (strlen(kTile[f->tile].name) != len || memcmp(kTile[f->tile].name, s, len) != 0))
        ++f->tile;
    if (f->tile == kTiles)
        return CONV_I8_ERR_PARAM;
    if (slash) {
        char *end;
        const long n = strtol(slash + 1, &end, 10);
        if (end == slash + 1 || *end || n < 1 || n > 64)
            return CONV_I8_ERR_PARAM;
        f->split = (int)n;
    }
    f->on = true;
    return CONV_I8_OK;
}

void set_plan(int64_t M, int64_t N, int64_t K, int es, int tile, int splits, GemmPlan *p)
{
    const int64_t nstages = ceil_div(K * es, kStageBytes);
    p->tile = tile;
    p->tiles_m = (int)ceil_div(M, kTile[tile].tm);
    p->tiles_n = (int)ceil_div(N, kTile[tile].tn);
    p->nstages = (int)nstages;
    p->kchunk = nstages > 0 ? (int)ceil_div(nstages, splits) : 0;
    p->splits = nstages > 0 ? (int)ceil_div(nstages, p->kchunk) : 1;
    p->part_ld = (int)round_up(N, 8);
    p->part_bytes = p->splits > 1 ? round_up((int64_t)p->splits * M * p->part_ld * 4, kWsAlign) : 0;
}

// The plan of a product of M rows whose first operand has two terms: partial sums of both.
void two_terms(int64_t M, GemmPlan *p)
{
    p->terms = 2;
    p->part_bytes = round_up(2 * (int64_t)p->splits * M * p->part_ld * 4, kWsAlign);
}

// Returns the microseconds expected.
double plan_gemm(int64_t M, int64_t N, int64_t K, int es, const Forced &forced, GemmPlan *p, const TileCost *costs = kCost)
{
    const int64_t nstages = ceil_div(K * es, kStageBytes);
    if (forced.on && forced.split > 0) {
        // of a product with fewer than four stages for each part, as many parts as have four
        const int64_t most = nstages / 4 > 1 ? nstages / 4 : 1;
        set_plan(M, N, K, es, forced.tile, (int)(forced.split < most ? forced.split : most), p);
        return gemm_cost(costs, forced.tile, M, N, K * es, p->splits);
    }
    int best = 0, best_s = 1;
    double least = 1e30;
    for (int t = 0; t < kTiles; ++t) {
        if (forced.on && t != forced.tile)
            continue;
        const int64_t tiles = ceil_div(M, kTile[t].tm) * ceil_div(N, kTile[t].tn);
        for (const int s : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
            // a split keeps eight stages, and two rounds of workgroups are enough
            if (s > 1 && (nstages < 8 * s || tiles * s > 2 * kCUs * kTile[t].occ))
                break;
            // a deep ring pays in the first round of workgroups only (2048x4096x512: two rounds
            // 16.3 us, 128x128 14.0)
            if (!forced.on && kTile[t].deep && tiles * s > kCUs)
                break;
            const double us = gemm_cost(costs, t, M, N, K * es, s);
            if (us < least) {
                least = us;
                best = t;
                best_s = s;
            }
        }
    }
    set_plan(M, N, K, es, best, best_s, p);
    return least;
}

bool grid_fits(const GemmPlan &p, int64_t M)
{
    return launch_fits((int64_t)p.tiles_m * p.tiles_n, 256) &&
           (!p.joined() || launch_fits(ceil_div(M * (p.part_ld / 8), 256), 256));
}

// C[M, N] = A B^T over K with the epilogue.  kbytes: inner bytes of a rows-form
// operand as stored (padded to 16).
GemmArgs gemm_args(const Operand &a, const void *ap, const Operand &b, const void *bp, int64_t M, int64_t N, int64_t K,
                   const GemmPlan &p, void *part, const Epilogue &epi)
{
    GemmArgs g;
    memset(&g, 0, sizeof g);
    g.a = (const uint8_t *)ap;
    g.b = (const uint8_t *)bp;
    g.lda = a.ld;
    g.ldb = b.ld;
    g.M = (int)M;
    g.N = (int)N;
    g.K = (int)K;
    g.kbytes = (int)round_up(K * a.es, 16);
    g.nstages = p.nstages;
    g.kchunk = p.kchunk;
    g.tiles_m = p.tiles_m;
    g.tiles_n = p.tiles_n;
    g.tiles = p.tiles_m * p.tiles_n;
    g.group = 8;
    g.part = p.joined() ? part : nullptr;
    g.part_ld = p.part_ld;
    g.part_stride = M * (int64_t)p.part_ld;
    g.epi = epi;
    // row strides (0 for an absent matrix) in elements of at most four bytes
    g.epi.tile_offsets = epi.ldo < (1 << 20) && epi.ldr < (1 << 20) && epi.ldp < (1 << 20);
    return g;
}

bool launch_gemm_of(int64_t dt, const Operand &a, const Operand &b, const GemmPlan &p, const GemmArgs &g, hipStream_t stream)
{
    return dt == DENSE_BF16 ? launch_gemm_bf16(p.tile, a.cols, b.cols, g, p.splits, stream)
         : dt == DENSE_FP16 ? launch_gemm_f16(p.tile, a.cols, b.cols, g, p.splits, stream)
         : dt == DENSE_E4M3 ? launch_gemm_f8e4(p.tile, g, p.splits, stream)
         : dt == DENSE_E5M2 ? launch_gemm_f8e5(p.tile, g, p.splits, stream)
                            : launch_gemm_i8(p.tile, a.cols, b.cols, g, p.splits, stream);
}

// a2: the first operand's second term, if the plan has two.
bool run_gemm(int64_t dt, const Operand &a, const Operand &b, const GemmPlan &p, const GemmArgs &g, hipStream_t stream,
              const void *a2 = nullptr)
{
    if (!launch_gemm_of(dt, a, b, p, g, stream))
        return false;
    if (!p.joined())
        return true;
    JoinArgs j = {p.splits, p.splits, 1.0f};
    if (p.terms > 1) {
        GemmArgs second = g;
        second.a = (const uint8_t *)a2;
        second.part = (float *)g.part + p.splits * g.part_stride;
        if (!launch_gemm_of(dt, a, b, p, second, stream))
            return false;
        j.copies = 2 * p.splits;
        j.scale = 1.0f / (dt == DENSE_BF16 ? second_term_up<bf16>() : second_term_up<f16>());
    }
    const int64_t items = (int64_t)g.M * (p.part_ld / 8);
    const dim3 grid((unsigned)ceil_div(items, 256)), block(256);
    if (dt == DENSE_INT8)
        hipLaunchKernelGGL(split_finish_kernel<true>, grid, block, 0, stream, g, j);
    else
        hipLaunchKernelGGL(split_finish_kernel<false>, grid, block, 0, stream, g, j);
    return hipGetLastError() == hipSuccess;
}

conv_i8_status_t check_workspace(const void *ws, size_t bytes, int64_t need)
{
    if (need == 0)
        return CONV_I8_OK;
    if (bytes < (size_t)need || ((uintptr_t)ws & (kWsAlign - 1)) != 0)
        return CONV_I8_ERR_WORKSPACE;
    return ws ? CONV_I8_OK : CONV_I8_ERR_NULL;
}

int describe(const GemmPlan &p, const Operand &a, const Operand &b, char *buf, size_t len)
{
    return snprintf(buf, len, "tile=%s tiles=%d split=%d stages=%d per_split=%d a=%s%s b=%s%s",
                    kTile[p.tile].name, p.tiles_m * p.tiles_n, p.splits, p.nstages, p.kchunk, a.cols ? "cols" : "rows", a.packed ? "_packed" : "",
                    b.cols ? "cols" : "rows", b.packed ? "_packed" : "");
}

}  // namespace
}  // namespace dense
