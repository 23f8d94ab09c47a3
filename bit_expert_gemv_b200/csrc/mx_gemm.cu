// Product of MXFP4 weights with MXFP8 tokens: y[t][r] = sum_c W[r][c] X[t][c].
//
// One kernel for every token count, on the block-scaled tensor-core
// instruction: 128 weight rows are the MMA's M, the tokens its N (16 to 256).
// The weights cross HBM packed; the TMA unit spreads each 16 nibbles over 16
// bytes of shared memory, which is the form the instruction takes, and the
// scales travel in 512-byte atoms that one copy brings into TMEM.  So no
// arithmetic instruction touches a weight: a few tokens are bound by the
// weights' stream from HBM, many by the tensor pipe.
//
// The kernel is persistent, one CTA per SM.  Roles (256 threads): warps 0 and 2
// fill a ring of stages (256 columns each) with weights and with tokens;
// warp 1 copies a stage's scales to TMEM and issues its eight MMAs; warps
// 4-7 read a tile's accumulators and write y while the next tile's MMAs run
// into the other accumulator buffer.  What a few instructions of one lane cost
// sets the pace of the rings: a turn of a producer's loop takes some 400 cycles
// (waiting for a stage, the copies' issue), which 128 columns of a stage did not
// cover.
//
// PAIR: two CTAs share a tile of 256 rows.  Either holds its own 128 rows and
// half of the tokens' bytes, so a CTA's shared memory takes in 24 KB instead of
// 40 KB per 128 x 128 x 256 products; the first CTA issues for both.  The second
// CTA's copies complete on the first one's barriers, which is what orders them
// before the MMAs that read them: a warp that waited for them and passed the news
// on would need a release at cluster scope for every stage.
//
// RESIDENT (up to 128 tokens, rows up to 8192 columns): the tokens' scales of all
// the CTA's columns are copied to TMEM once.  Copying them with every stage cost
// the issuing warp 14 % at one token, where its instructions set the pace.
//
// Without PAIR, the tiles that are left after whole rounds are split over the
// columns by a cluster of up to 8 CTAs, whose partial sums are added through
// distributed shared memory in rank order.
#include <atomic>

#include "mx.cuh"
#include "tc_mx.cuh"
#include "tma.cuh"

namespace gale {
namespace {

constexpr int kGThreads = 256;
constexpr int kGK = 2;                           // column tiles of a stage
constexpr int kGABytes = kMxTile * kMxTile;      // weights of a column tile: 128 rows x 128 columns, a byte each
constexpr int kGMaxStages = 8;
constexpr int kGMaxShared = 96;                  // columns that the two accumulator buffers may share
constexpr int kGMaxN = 256;
constexpr int kGSmemSm = 226 * 1024;             // dynamic shared memory a CTA can have (1 KB for the barriers)

struct GemmArgs {
    const uint8_t* wsc;     // scale atoms of W [row tiles][nt][512]
    const uint8_t* xsc;     // scale atoms of X
    void* y;
    int32_t* status;
    int64_t rows, tokens, ldy;
    int nt;                 // column tiles
    int rtiles;             // 128-row tiles
    int n;                  // tokens of a tile (the MMA's N)
    int ntt;                // token tiles
    int tiles;              // row tiles (of 256 rows with PAIR) x token tiles
    int xatoms;             // scale atoms a token tile can touch
    int sfcols;             // TMEM columns of a stage's scales: per column tile 4 (W) and 4 per atom (X)
    int workers;            // CTAs (pairs with PAIR) that take whole tiles
    int whole;              // tiles that each worker takes whole (the last one may be missing when split is 1)
    int split;              // CTAs that share a left-over tile (the cluster)
    int joint;              // left-over tiles of a cluster, at most
    int stages;
    int stage_bytes;
    int res_off;            // RESIDENT: the tokens' scales in shared memory
    int res_col;            // and in TMEM
    int cols;               // TMEM columns
    int d1;                 // TMEM column of the second accumulator buffer
    int ydtype;
    int pair16;             // 16-bit y may be written two rows at a time
};

// Unit u of this CTA: a tile and a range of its column tiles.
struct GemmUnit {
    int rt, tt, k0, k1;
    bool joint;
};
template <bool PAIR>
__device__ __forceinline__ bool gemm_unit(const GemmArgs& a, int u, GemmUnit& w) {
    const int worker = PAIR ? blockIdx.x >> 1 : blockIdx.x;
    int tile;
    if (u < a.whole) {
        tile = u * a.workers + worker;
        w.k0 = 0;
        w.k1 = a.nt;
        w.joint = false;
    } else {
        if (PAIR || u >= a.whole + a.joint) return false;
        const int cluster = blockIdx.x / a.split, part = blockIdx.x % a.split;
        tile = a.whole * a.workers + cluster + (u - a.whole) * (a.workers / a.split);
        const int pieces = (a.nt + kGK - 1) / kGK;
        w.k0 = pieces * part / a.split * kGK;
        w.k1 = min(pieces * (part + 1) / a.split * kGK, a.nt);
        w.joint = true;
    }
    if (tile >= a.tiles) return false;
    w.rt = tile / a.ntt;
    w.tt = tile % a.ntt;
    return true;
}

// The column tiles that this CTA's units cover.
template <bool PAIR>
__device__ __forceinline__ void gemm_columns(const GemmArgs& a, int& k0, int& k1) {
    k0 = 0;
    k1 = a.nt;
    GemmUnit w;
    if (a.whole == 0 && gemm_unit<PAIR>(a, 0, w)) {
        k0 = w.k0;
        k1 = w.k1;
    }
}

// 16 tokens of one row per lane to y; `full`: all of the warp's rows exist.
__device__ __forceinline__ void gemm_store16(const GemmArgs& a, int64_t t, int64_t row, int lane, bool full,
                                             const float (&v)[16]) {
    if (a.ydtype == GALE_F32) {
        float* y = static_cast<float*>(a.y) + t * a.ldy + row;
        if (full && t + 16 <= a.tokens) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                *y = v[i];
                y += a.ldy;
            }
        } else if (row < a.rows) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (t + i < a.tokens) *y = v[i];
                y += a.ldy;
            }
        }
    } else if (a.pair16) {
        // lanes 2i and 2i + 1 trade values so that each writes two rows of one of two tokens
        const int odd = lane & 1;
        const int64_t r0 = row - odd;
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const float got = __shfl_xor_sync(0xffffffffu, odd ? v[i] : v[i + 1], 1);
            w[i / 2] = pack16(a.ydtype, odd ? got : v[i], odd ? v[i + 1] : got);
        }
        uint16_t* y = static_cast<uint16_t*>(a.y) + (t + odd) * a.ldy + r0;
        if (full && t + 16 <= a.tokens) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                *reinterpret_cast<uint32_t*>(y) = w[i];
                y += 2 * a.ldy;
            }
        } else if (r0 < a.rows) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (t + 2 * i + odd < a.tokens) {
                    if (r0 + 1 < a.rows) *reinterpret_cast<uint32_t*>(y) = w[i];
                    else *y = uint16_t(w[i]);
                }
                y += 2 * a.ldy;
            }
        }
    } else if (row < a.rows) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (t + i < a.tokens) store_rn(a.y, a.ydtype, (t + i) * a.ldy + row, v[i]);
    }
}

// Four rows of one token, the first of them row r, to y.
__device__ __forceinline__ void gemm_store4(const GemmArgs& a, int64_t t, int64_t r, const float4& v) {
    const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (r + i < a.rows) store_rn(a.y, a.ydtype, t * a.ldy + r + i, f[i]);
}

// Adds the cluster's partial sums of one left-over tile, four rows at a time.
template <int SPLIT>
__device__ __forceinline__ void gemm_join(const GemmArgs& a, const GemmUnit& w, uint32_t at, int part) {
    const int64_t t0 = int64_t(w.tt) * a.n;
    const int live = int(min(int64_t(a.n), a.tokens - t0)) * (kMxTile / 4);
#pragma unroll 2
    for (int i = part * kGThreads + threadIdx.x; i < live; i += SPLIT * kGThreads) {
        float4 p[SPLIT];
#pragma unroll
        for (int q = 0; q < SPLIT; ++q) p[q] = ld_cluster_f4(at + i * 16, q);
        float4 v = p[0];
#pragma unroll
        for (int q = 1; q < SPLIT; ++q) {
            v.x += p[q].x;
            v.y += p[q].y;
            v.z += p[q].z;
            v.w += p[q].w;
        }
        gemm_store4(a, t0 + i / (kMxTile / 4), int64_t(w.rt) * kMxTile + i % (kMxTile / 4) * 4, v);
    }
}

template <bool PAIR, bool RESIDENT>
__global__ void __launch_bounds__(kGThreads, 1) mx_gemm_kernel(const __grid_constant__ CUtensorMap wmap,
                                                              const __grid_constant__ CUtensorMap xmap,
                                                              const __grid_constant__ CUtensorMap wscmap,
                                                              const __grid_constant__ CUtensorMap xscmap,
                                                              const __grid_constant__ GemmArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_align1024(smem_raw);
    // full: a stage's bytes are here, and in the pair's other CTA (two producers; of a pair the first CTA's
    // alone is used); empty: its MMAs are done; acc_full: a unit's accumulators are final; acc_free: the columns
    // that the next unit's buffer shares with them have been read
    __shared__ uint64_t full[kGMaxStages], empty[kGMaxStages], acc_full[2], acc_free, res_full;
    __shared__ uint32_t tmem_base;
    const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
    const int rank = PAIR ? int(blockIdx.x & 1) : 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(&full[s], 2);
            mbar_init(&empty[s], 1);
        }
        mbar_init(&acc_full[0], 1);
        mbar_init(&acc_full[1], 1);
        mbar_init(&acc_free, PAIR ? 8 : 4);
        if (RESIDENT) mbar_init(&res_full, 1);
        fence_mbar_init();
    }
    if (warp == 3) {
        if (lane == 0) {
            prefetch_tensormap(&wmap);
            prefetch_tensormap(&xmap);
            if (PAIR) {
                prefetch_tensormap(&wscmap);
                prefetch_tensormap(&xscmap);
            }
        }
        __syncwarp();
        if (PAIR) {
            tmem_alloc_pair(&tmem_base, a.cols);
        } else {
            tmem_alloc(&tmem_base, a.cols);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();      // the other CTA's barriers are ready too
    tc_fence_after();
    pdl_wait();                    // the kernels before this one are done: from here on memory is read and written
    const uint32_t tmem = tmem_base;
    const int xrows = PAIR ? a.n / 2 : a.n;      // tokens whose bytes this CTA holds
    const int xbytes = xrows * kMxTile;
    bool ok = true;
    GemmUnit w;
    const uint32_t ring = smem_u32(smem), ring_end = ring + a.stages * a.stage_bytes;
    const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty);
    if (warp == 0 || warp == 2) {
        const bool lead = elect_one();
        int issued = 0;
        // (st, s8: the stage's shared memory and the offset of its barriers)
        uint32_t st = ring, s8 = 0, phase = 1;      // of the empty barriers: the first turn of the ring passes
        const int atoms_all = int((a.tokens + kMxTile - 1) / kMxTile);
        const uint32_t landed0 = PAIR ? cluster_address(full0, 0) : full0;      // where the copies complete
        if (RESIDENT && warp == 2) {
            int k0, k1;
            gemm_columns<PAIR>(a, k0, k1);
            mbar_expect_lead(lead, smem_u32(&res_full), (k1 - k0) * kMxAtomBytes);
            bulk_load_lead(lead, ring + a.res_off, a.xsc + int64_t(k0) * kMxAtomBytes, (k1 - k0) * kMxAtomBytes,
                           smem_u32(&res_full));
        }
        for (int u = 0; ok && gemm_unit<PAIR>(a, u, w); ++u) {
            const int t0 = w.tt * a.n;
            const int atom0 = t0 / kMxTile;
            const int atoms = RESIDENT ? 0 : min(a.xatoms, atoms_all - atom0);
            const int rt = PAIR ? 2 * w.rt + rank : w.rt;
            // (a pair's second row tile may not exist: its lines read as zero, its scales are the last tile's)
            const uint8_t* wsc = a.wsc + int64_t(min(rt, a.rtiles - 1)) * a.nt * kMxAtomBytes;
            const uint8_t* xsc = a.xsc + int64_t(atom0) * a.nt * kMxAtomBytes;
            const int line = rt * a.nt * kMxTile;
            for (int k = w.k0; k < w.k1; k += kGK) {
                ok = mbar_wait_warp<PAIR>(empty0 + s8, phase);
                if (!ok) break;
                const int kt = min(kGK, w.k1 - k);
                const uint32_t bar = full0 + s8;
                const uint32_t sc = st + kGK * (kGABytes + xbytes);
                if (PAIR && warp == 0) {
                    // (the first CTA expects the bytes of both; scales come two atoms at a time)
                    if (rank == 0)
                        mbar_expect_lead(lead, bar, 2 * (kt * kMx4TileBytes + kGK * kMxAtomBytes));
                    tma_load_2d_pair(lead, st, &wmap, landed0 + s8, 0, line + k * kMxTile);
                    if (kt == 2)
                        tma_load_2d_pair(lead, st + kGABytes, &wmap, landed0 + s8, 0, line + (k + 1) * kMxTile);
                    tma_load_2d_pair(lead, sc, &wscmap, landed0 + s8, 0, min(rt, a.rtiles - 1) * a.nt + k);
                } else if (PAIR) {
                    const uint32_t xs = st + kGK * kGABytes;
                    if (rank == 0)
                        mbar_expect_lead(lead, bar, 2 * (kt * xbytes + atoms * kGK * kMxAtomBytes));
                    tma_load_2d_pair(lead, xs, &xmap, landed0 + s8, k * kMxTile, t0 + rank * xrows);
                    if (kt == 2)
                        tma_load_2d_pair(lead, xs + xbytes, &xmap, landed0 + s8, (k + 1) * kMxTile, t0 + rank * xrows);
                    for (int j = 0; j < atoms; ++j)
                        tma_load_2d_pair(lead, sc + (1 + j) * kGK * kMxAtomBytes, &xscmap, landed0 + s8, 0,
                                         (atom0 + j) * a.nt + k);
                } else if (warp == 0) {
                    // the spread weights count with their packed bytes
                    mbar_expect_lead(lead, bar, kt * (kMx4TileBytes + kMxAtomBytes));
                    tma_load_2d(lead, st, &wmap, bar, 0, line + k * kMxTile);
                    if (kt == 2) tma_load_2d(lead, st + kGABytes, &wmap, bar, 0, line + (k + 1) * kMxTile);
                    bulk_load_lead(lead, sc, wsc + k * kMxAtomBytes, kt * kMxAtomBytes, bar);
                } else {
                    const uint32_t xs = st + kGK * kGABytes;
                    mbar_expect_lead(lead, bar, kt * (xbytes + atoms * kMxAtomBytes));
                    tma_load_2d(lead, xs, &xmap, bar, k * kMxTile, t0);
                    if (kt == 2) tma_load_2d(lead, xs + xbytes, &xmap, bar, (k + 1) * kMxTile, t0);
                    for (int j = 0; j < atoms; ++j)
                        bulk_load_lead(lead, sc + (1 + j) * kGK * kMxAtomBytes,
                                       xsc + (int64_t(j) * a.nt + k) * kMxAtomBytes, kt * kMxAtomBytes, bar);
                }
                ++issued;
                st += a.stage_bytes;
                s8 += 8;
                if (st == ring_end) {
                    st = ring;
                    s8 = 0;
                    phase ^= 1;
                }
            }
        }
        // before the CTA may end (bounded): the last stages' MMAs have reported, or after a failure the last
        // copies have landed (a pair's first CTA waits for both CTAs', the second one for it at the cluster's barrier)
        for (int i = max(0, issued - a.stages); i < issued && (!PAIR || rank == 0 || ok); ++i)
            ok = mbar_wait_warp<PAIR>((ok ? empty0 : full0) + i % a.stages * 8, (i / a.stages) & 1) && ok;
    } else if (warp == 1 && (!PAIR || rank == 0)) {
        const bool lead = elect_one();
        const uint32_t idesc = umma_idesc_mx(PAIR ? 2 * kMxTile : kMxTile, a.n);
        const uint32_t sf_first = tmem + a.cols - a.stages * a.sfcols;
        const uint64_t xstep = xbytes >> 4;
        int kres = 0;
        if (RESIDENT) {
            int k1;
            gemm_columns<PAIR>(a, kres, k1);
            ok = mbar_wait_warp(smem_u32(&res_full), 0);
            if (ok) {
                tc_fence_after();
                for (int k = kres; k < k1; ++k)
                    tmem_copy_scales(lead, tmem + a.res_col + 4 * (k - kres),
                                     scale_atom_desc(ring + a.res_off + (k - kres) * kMxAtomBytes));
            }
        }
        // scale copies of a stage, and their TMEM columns per column tile
        const int ncopy = RESIDENT ? 1 : 1 + a.xatoms;
        uint32_t st = ring, s8 = 0, phase = 0, sf = sf_first;
        for (int u = 0; ok && gemm_unit<PAIR>(a, u, w); ++u) {
            const uint32_t d = tmem + ((u & 1) ? a.d1 : 0);
            const uint32_t xoff = 4 + ((w.tt * a.n) % kMxTile) / 32;      // scale column of the tile's first token
            if (u > 0) {
                ok = mbar_wait_warp<PAIR>(smem_u32(&acc_free), (u - 1) & 1);
                if (!ok) break;
                tc_fence_after();
            }
            for (int k = w.k0; k < w.k1; k += kGK) {
                ok = mbar_wait_warp<PAIR>(full0 + s8, phase);
                if (!ok) break;
                tc_fence_after();
                const int kt = min(kGK, w.k1 - k);
                const uint64_t from = scale_atom_desc(st + kGK * (kGABytes + xbytes));
                const uint64_t ad = umma_desc_sw128(st), bd = umma_desc_sw128(st + kGK * kGABytes);
#pragma unroll
                for (int j = 0; j < kGK; ++j) {
                    if (j == kt) break;
                    const uint32_t sfj = sf + j * 4 * ncopy;
                    for (int i = 0; i < ncopy; ++i) {
                        if (PAIR) tmem_copy_scales_pair(lead, sfj + 4 * i, from + (i * kGK + j) * (kMxAtomBytes >> 4));
                        else tmem_copy_scales(lead, sfj + 4 * i, from + (i * kGK + j) * (kMxAtomBytes >> 4));
                    }
                }
#pragma unroll
                for (int j = 0; j < kGK; ++j) {
                    if (j == kt) break;
                    const uint32_t sfj = sf + j * 4 * ncopy;
                    const uint32_t sfx = RESIDENT ? tmem + a.res_col + 4 * (k + j - kres) : sfj + xoff;
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const uint32_t more = (k > w.k0 || j > 0 || b > 0) ? 1u : 0u;
                        const uint32_t id = umma_idesc_scale_id(idesc, b);
                        const uint64_t aj = ad + j * (kGABytes >> 4) + 2 * b, bj = bd + j * xstep + 2 * b;
                        if (PAIR) umma_mx_pair(lead, d, aj, bj, id, sfj, sfx, more);
                        else umma_mx(lead, d, aj, bj, id, sfj, sfx, more);
                    }
                }
                if (PAIR) umma_commit_pair(lead, &empty[0] + (s8 >> 3));
                else umma_commit_one(lead, &empty[0] + (s8 >> 3));
                st += a.stage_bytes;
                s8 += 8;
                sf += a.sfcols;
                if (st == ring_end) {
                    st = ring;
                    s8 = 0;
                    sf = sf_first;
                    phase ^= 1;
                }
            }
            if (PAIR) umma_commit_pair(lead, &acc_full[u & 1]);
            else umma_commit_one(lead, &acc_full[u & 1]);
        }
    } else if (warp >= 4) {
        const int quarter = warp & 3;
        const uint32_t lanes = uint32_t(quarter) << 21;
        for (int u = 0; ok && gemm_unit<PAIR>(a, u, w); ++u) {
            ok = mbar_wait_warp<PAIR>(smem_u32(&acc_full[u & 1]), (u >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = tmem + lanes + ((u & 1) ? a.d1 : 0);
            const int64_t row = int64_t(PAIR ? 2 * w.rt + rank : w.rt) * kMxTile + quarter * 32 + lane;
            const bool rows_full = row - lane + 32 <= a.rows;
            float* ps = nullptr;
            if (w.joint)     // partial sums [token][128 rows] over the ring (the last unit) or behind it
                ps = reinterpret_cast<float*>(smem + (a.joint > 1 ? int64_t(a.stages) * a.stage_bytes : 0)) +
                     int64_t(u - a.whole) * a.n * kMxTile + quarter * 32 + lane;
            const int64_t t0 = int64_t(w.tt) * a.n;
            auto put = [&](int c, const float (&v)[16]) {
                if (ps) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) ps[(c + i) * kMxTile] = v[i];
                } else if (t0 + c < a.tokens) {
                    gemm_store16(a, t0 + c, row, lane, rows_full, v);
                }
            };
            auto release = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR && rank) mbar_arrive_cluster(smem_u32(&acc_free), 0);
                    else mbar_arrive(&acc_free);
                }
            };
            // the columns that the other buffer shares (the last n - d1 of buffer 0, the first of buffer 1) go
            // to registers first, so that the next unit's MMAs wait for no store
            const int shared = a.n - a.d1;
            const int c0 = (u & 1) ? 0 : a.d1;
            if (shared > 0) {
                float v[kGMaxShared / 16][16];
#pragma unroll
                for (int q = 0; q < kGMaxShared / 16; ++q)
                    if (16 * q < shared) tmem_ld16_start(d + c0 + 16 * q, v[q]);
                tmem_wait_ld();
                release();
#pragma unroll
                for (int q = 0; q < kGMaxShared / 16; ++q)
                    if (16 * q < shared) put(c0 + 16 * q, v[q]);
            } else {
                release();
            }
            const int c1 = (u & 1) ? max(shared, 0) : 0, c2 = (u & 1) ? a.n : min(a.n, a.d1);
            for (int c = c1; c < c2; c += 16) {
                float v[16];
                tmem_ld16(d + c, v);
                put(c, v);
            }
        }
    }
    if (!ok) set_status(a.status, GALE_ERR_TIMEOUT);
    if (!PAIR && a.split > 1) {
        cluster_sync();
        const int part = blockIdx.x % a.split;
        uint32_t at = smem_u32(smem) + (a.joint > 1 ? a.stages * a.stage_bytes : 0);
        for (int u = a.whole; gemm_unit<PAIR>(a, u, w); ++u, at += a.n * kMxTile * 4) {
            if (a.split == 2) gemm_join<2>(a, w, at, part);
            else if (a.split == 4) gemm_join<4>(a, w, at, part);
            else gemm_join<8>(a, w, at, part);
        }
    }
    tc_fence_before();
    __syncthreads();
    // nobody reads a peer's partial sums, reads its operands or arrives on its barriers after this (reads have
    // returned when their values were used; arrivals need the release)
    if (PAIR) cluster_sync();
    else if (a.split > 1) cluster_sync_relaxed();
    if (warp == 3) {
        tc_fence_after();
        if (PAIR) tmem_dealloc_pair(tmem, a.cols);
        else tmem_dealloc(tmem, a.cols);
    }
}

struct GemmPlan {
    GemmArgs a;
    bool pair, resident;
    int grid, smem;
};

// Clusters of `size` CTAs of this kernel that the device holds at once (an SM
// that is left over in its group of SMs holds none of a larger cluster).
int gemm_clusters(int size) {
    static std::atomic<int> found[64][4];       // per device, by log2 of the size: an attribute of the device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    const int slot = size == 1 ? 0 : size == 2 ? 1 : size == 4 ? 2 : 3;
    int n = found[dev][slot];
    if (!n) {
        if (ensure_smem(reinterpret_cast<const void*>(mx_gemm_kernel<false, false>), kGSmemSm) != GALE_OK) return 0;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(unsigned(size) * 16);
        cfg.blockDim = dim3(kGThreads);
        cfg.dynamicSmemBytes = kGSmemSm;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim = {unsigned(size), 1, 1};
        cfg.attrs = at;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, mx_gemm_kernel<false, false>, &cfg) != cudaSuccess) {
            cudaGetLastError();
            return 0;
        }
        found[dev][slot] = n;
    }
    return n;
}

// Chooses the tile's tokens, pairs or single CTAs and the split of left-over tiles
// by an estimate in cycles.  A stage of 256 columns takes 4 n + 64 (the tensor
// pipe), 640 (its issue) or its bytes at 64 a cycle, whichever is longest; a unit
// some 300 more, 800 from 192 tokens on, 1000 where its accumulators share columns
// with the last unit's; a join 1500 and 25 a token.  What counts is the sum of the
// longest CTA's time and the average one's: many tokens are bound by power, and
// what idles lets the others run faster.  (1000 tokens x [5000 x 4000]: 192-token
// pairs 27 us, 256-token pairs 32 us; 4096 x [4096 x 4096]: 58 and 54 us.)  False
// if the device does not answer.
bool gemm_plan(int64_t rows, int nt, int64_t tokens, GemmPlan& p) {
    GemmArgs& a = p.a;
    a.rows = rows;
    a.tokens = tokens;
    a.nt = nt;
    a.rtiles = int((rows + kMxTile - 1) / kMxTile);
    const int pieces = (nt + kGK - 1) / kGK;
    int64_t best = INT64_MAX;
    int join_bytes = 0;
    auto consider = [&](bool pair, int n, int split) {
        const int clusters = gemm_clusters(pair ? 2 : split);
        if (clusters < 1) return false;
        const int ntt = int((tokens + n - 1) / n);
        const int tiles = (pair ? (a.rtiles + 1) / 2 : a.rtiles) * ntt;
        const int workers = pair ? clusters : clusters * split;
        const bool joins = !pair && split > 1;
        const int whole = joins ? tiles / workers : (tiles + workers - 1) / workers;
        const int left = joins ? tiles - whole * workers : 0;
        const int joint = (left + clusters - 1) / clusters;
        if (joins && (joint == 0 || pieces < 2 * split)) return true;
        const int64_t bytes = joint > 1 ? int64_t(joint) * n * kMxTile * 4 : 0;
        if (bytes > 64 * 1024) return true;
        const int64_t load = 2 * (kMx4TileBytes + kMxAtomBytes) + (pair ? n : 2 * n) * int64_t(kMxTile + 4);
        int64_t step = 4 * n + 64 > 640 ? 4 * n + 64 : 640;
        if (load / 64 > step) step = load / 64;
        const int64_t unit = n > 208 ? 1000 : n >= 192 ? 800 : 300;
        const int64_t tile = pieces * step + unit;
        const int64_t longest = whole * tile + joint * (((pieces + split - 1) / split) * step + unit) +
                                (joint ? 1500 + 25 * n : 0);
        const int64_t cost = longest + tiles * tile / workers + (pair ? 1000 : 0);
        if (cost < best) {
            best = cost;
            p.pair = pair;
            a.n = n;
            a.ntt = ntt;
            a.tiles = tiles;
            a.split = joins ? split : 1;
            a.workers = workers;
            a.whole = whole;
            a.joint = joint;
            join_bytes = int(bytes);
        }
        return true;
    };
    // one tile for all tokens (the MMA's N in steps of 16, of 32 over a pair), or tiles of a multiple of 64 (a
    // tile's first scale sits at an even TMEM column)
    const int all = tokens <= kGMaxN ? int(align_up(tokens, 16)) : 0;
    for (int i = 0; i <= kGMaxN / 64; ++i) {
        const int n = i == 0 ? all : 64 * i;
        if (n == 0 || (i > 0 && all > 0 && n >= all)) continue;
        for (int s = 1; s <= 8; s *= 2)
            if (!consider(false, n, s)) return false;
        if (n % 32 == 0 && n >= 64 && !consider(true, n, 1)) return false;
    }
    if (p.pair || a.split == 1) {
        if (a.workers > a.tiles) a.workers = a.tiles;
    } else if (a.whole == 0 && a.tiles < a.workers / a.split) {
        a.workers = a.tiles * a.split;      // clusters without a tile are not launched
    }
    p.grid = p.pair ? 2 * a.workers : a.workers;
    // tokens t0 .. t0 + n - 1 of a tile that starts at a multiple of n
    a.xatoms = a.ntt == 1 ? (a.n + kMxTile - 1) / kMxTile : a.n % kMxTile == 0 ? a.n / kMxTile : a.n / kMxTile + 2;
    if (a.xatoms > 3) a.xatoms = 3;
    const int xrows = p.pair ? a.n / 2 : a.n;
    p.resident = !p.pair && a.ntt == 1 && a.xatoms == 1 && nt <= 64;
    const int ncopy = p.resident ? 1 : 1 + a.xatoms;
    const int res_bytes = p.resident ? int(align_up((a.whole ? nt : (nt + a.split - 1) / a.split + kGK) * kMxAtomBytes, 1024)) : 0;
    a.stage_bytes = int(align_up(kGK * (kGABytes + xrows * kMxTile + kMxAtomBytes * ncopy), 1024));
    a.stages = (kGSmemSm - 1024 - join_bytes - res_bytes) / a.stage_bytes;
    if (a.stages > kGMaxStages) a.stages = kGMaxStages;
    a.res_off = a.stages * a.stage_bytes + join_bytes;
    a.sfcols = kGK * 4 * ncopy;
    const int res_cols = p.resident ? 4 * nt : 0;
    const int units = a.whole + a.joint;
    int cols = 32;
    while (cols < (units > 1 ? 2 : 1) * a.n + a.stages * a.sfcols + res_cols && cols < 512) cols *= 2;
    a.cols = cols;
    const int avail = (cols - a.stages * a.sfcols - res_cols) / 16 * 16;
    a.d1 = units == 1 || avail >= 2 * a.n ? a.n : avail - a.n;
    a.res_col = cols - a.stages * a.sfcols - res_cols;
    p.smem = a.stages * a.stage_bytes + join_bytes + res_bytes + 1024;
    // As large a share of the SM's shared memory as of its TMEM, so that a CTA
    // that is resident never waits for TMEM columns.
    const int least = int(int64_t(kGSmemSm) * cols / 512);
    if (p.smem < least) p.smem = least;
    return a.n - a.d1 <= kGMaxShared;
}

}  // namespace
}  // namespace gale

extern "C" size_t gale_mx_gemm_workspace_size(int64_t rows, int64_t cols, int64_t tokens) {
    gale_mx_layout_t L;
    if (gale_mx4_layout(rows, cols, &L) != GALE_OK || gale_mx8_layout(tokens, cols, &L) != GALE_OK) return 0;
    return 256;   // the status word
}

extern "C" int gale_mx_gemm(const void* w4, int64_t rows, int64_t cols, const void* x8, int64_t tokens, void* y,
                            int y_dtype, int64_t ldy, void* ws, size_t ws_bytes, void* stream) {
    using namespace gale;
    gale_mx_layout_t W, X;
    if (!valid_dtype(y_dtype) || gale_mx4_layout(rows, cols, &W) != GALE_OK || tokens < 0) return GALE_ERR_ARG;
    if (tokens == 0) return GALE_OK;
    if (gale_mx8_layout(tokens, cols, &X) != GALE_OK || !w4 || !x8 || !y || ldy < rows) return GALE_ERR_ARG;
    if (!aligned(w4, 256) || !aligned(x8, 256) || !aligned(y, dtype_size(y_dtype))) return GALE_ERR_ALIGN;
    if (!ws || ws_bytes < gale_mx_gemm_workspace_size(rows, cols, tokens)) return GALE_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return GALE_ERR_ALIGN;
    const uint8_t* w = static_cast<const uint8_t*>(w4);
    const uint8_t* x = static_cast<const uint8_t*>(x8);
    if (rows * tokens > (int64_t(1) << 42)) return GALE_ERR_UNSUPPORTED;   // (tiles are counted in 32 bits)
    GemmPlan p{};
    if (!gemm_plan(rows, int(W.cols_padded / kMxTile), tokens, p)) return GALE_ERR_CUDA;
    p.a.wsc = w + W.s_offset;
    p.a.xsc = x + X.s_offset;
    p.a.y = y;
    p.a.status = static_cast<int32_t*>(ws);
    p.a.ldy = ldy;
    p.a.ydtype = y_dtype;
    CUtensorMap wmap, xmap, wscmap{}, xscmap{};      // (the scales' maps: pairs only)
    int rc = make_map_mx4(&wmap, w, W.q_bytes / (kMxTile / 2));
    if (rc == GALE_OK) rc = make_map_bytes(&xmap, x, W.cols_padded, tokens, kMxTile, p.pair ? p.a.n / 2 : p.a.n);
    if (rc == GALE_OK && p.pair) rc = make_map_atoms(&wscmap, p.a.wsc, W.s_bytes / kMxAtomBytes);
    if (rc == GALE_OK && p.pair) rc = make_map_atoms(&xscmap, p.a.xsc, X.s_bytes / kMxAtomBytes);
    if (rc != GALE_OK) return rc;
    p.a.pair16 = ldy % 2 == 0 && aligned(y, 4);
    auto kern = p.pair ? mx_gemm_kernel<true, false> : p.resident ? mx_gemm_kernel<false, true> : mx_gemm_kernel<false, false>;
    if (ensure_smem(reinterpret_cast<const void*>(kern), p.smem) != GALE_OK) return GALE_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(p.grid));
    cfg.blockDim = dim3(kGThreads);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = as_stream(stream);
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {unsigned(p.pair ? 2 : p.a.split), 1, 1};
    // its set-up may run while the kernel before it ends (the kernel waits for that before it touches memory)
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kern, wmap, xmap, wscmap, xscmap, p.a) != cudaSuccess) {
        cudaGetLastError();      // reported here, not by the next call
        return GALE_ERR_CUDA;
    }
    return GALE_OK;
}
