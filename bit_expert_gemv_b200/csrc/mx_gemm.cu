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
// Roles (192 threads): warp 0 fills a ring of stages (128 columns each) by TMA;
// one lane of warp 1 copies the stage's scales to TMEM and issues its four
// MMAs; warps 2-5 read the accumulators and write y.  Where there are fewer
// tiles than SMs, a cluster of 2 to 8 CTAs splits the columns of one tile and
// adds the partial sums through distributed shared memory, in rank order.
#include "mx.cuh"
#include "tc_mx.cuh"
#include "tma.cuh"

namespace gale {
namespace {

constexpr int kGThreads = 192;
constexpr int kGABytes = kMxTile * kMxTile;      // a stage's weights: 128 rows x 128 columns, a byte each
constexpr int kGMaxStages = 8;
constexpr int kGSfCols = 16;                     // TMEM columns of a stage's scales: 4 (W) + up to 12 (X)
constexpr int kGMaxN = 256;
constexpr int kGSmemSm = 226 * 1024;             // dynamic shared memory a CTA can have (1 KB for the barriers)

struct GemmArgs {
    const uint8_t* wsc;     // scale atoms of W [row tiles][nt][512]
    const uint8_t* xsc;     // scale atoms of X
    void* y;
    int32_t* status;
    int64_t rows, tokens, ldy;
    int nt;                 // column tiles
    int n;                  // tokens of a tile (the MMA's N)
    int ntt;                // token tiles
    int xatoms;             // scale atoms a token tile can touch
    int split;              // CTAs per tile (the cluster)
    int stages;
    int stage_bytes;
    int cols;               // TMEM columns
    int ydtype;
};

__global__ void __launch_bounds__(kGThreads) mx_gemm_kernel(const __grid_constant__ CUtensorMap wmap,
                                                           const __grid_constant__ CUtensorMap xmap, GemmArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_align1024(smem_raw);
    __shared__ uint64_t full[kGMaxStages], empty[kGMaxStages], accum;
    __shared__ uint32_t tmem_base;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile = blockIdx.x / a.split, part = blockIdx.x % a.split;
    const int rt = tile / a.ntt, tt = tile % a.ntt;
    const int t0 = tt * a.n;
    const int k0 = int(int64_t(a.nt) * part / a.split), k1 = int(int64_t(a.nt) * (part + 1) / a.split);
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(&accum, 1);
        fence_mbar_init();
        prefetch_tensormap(&wmap);
        prefetch_tensormap(&xmap);
    }
    if (warp == 1) {
        tmem_alloc(&tmem_base, a.cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    const int xbytes = a.n * kMxTile;
    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {
            const int atom0 = t0 / kMxTile;
            const int atoms_all = int((a.tokens + kMxTile - 1) / kMxTile);
            const int atoms = min(a.xatoms, atoms_all - atom0);
            // (the spread weights count with their packed bytes)
            const uint32_t tx = uint32_t(kMx4TileBytes + xbytes + kMxAtomBytes * (1 + atoms));
            int k = k0;
            for (; k < k1; ++k) {
                const int s = (k - k0) % a.stages, round = (k - k0) / a.stages;
                if (round > 0) ok = mbar_wait(&empty[s], (round - 1) & 1);
                if (!ok) break;
                uint8_t* st = smem + int64_t(s) * a.stage_bytes;
                mbar_arrive_expect_tx(&full[s], tx);
                tma_load_2d(st, &wmap, &full[s], 0, (rt * a.nt + k) * kMxTile);
                tma_load_2d(st + kGABytes, &xmap, &full[s], k * kMxTile, t0);
                uint8_t* sc = st + kGABytes + xbytes;
                bulk_load(sc, a.wsc + (int64_t(rt) * a.nt + k) * kMxAtomBytes, kMxAtomBytes, &full[s]);
                for (int i = 0; i < atoms; ++i)
                    bulk_load(sc + (1 + i) * kMxAtomBytes, a.xsc + (int64_t(atom0 + i) * a.nt + k) * kMxAtomBytes,
                              kMxAtomBytes, &full[s]);
            }
            if (!ok)      // copies in flight land before the CTA ends (bounded)
                for (int j = max(k0, k - a.stages); j < k; ++j)
                    mbar_wait(&full[(j - k0) % a.stages], ((j - k0) / a.stages) & 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = umma_idesc_mx(kMxTile, a.n);
            const uint32_t sf_first = tmem + a.cols - a.stages * kGSfCols;
            const uint32_t xoff = 4 + (t0 % kMxTile) / 32;      // first scale column of the tile's first token
            for (int k = k0; k < k1 && ok; ++k) {
                const int s = (k - k0) % a.stages, round = (k - k0) / a.stages;
                ok = mbar_wait(&full[s], round & 1);
                if (!ok) break;
                tc_fence_after();
                const uint32_t st = smem_u32(smem + int64_t(s) * a.stage_bytes);
                const uint32_t sc = st + kGABytes + xbytes;
                const uint32_t sf = sf_first + s * kGSfCols;
                for (int i = 0; i <= a.xatoms; ++i)
                    tmem_copy_scales(sf + 4 * i, scale_atom_desc(sc + i * kMxAtomBytes));
                const uint64_t ad = umma_desc_sw128(st), bd = umma_desc_sw128(st + kGABytes);
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    umma_mx(tmem, ad + 2 * b, bd + 2 * b, umma_idesc_scale_id(idesc, b), sf, sf + xoff,
                            (k > k0 || b > 0) ? 1u : 0u);
                umma_commit(&empty[s]);
            }
            umma_commit(&accum);
        }
        __syncwarp();
    }
    // (the accumulators are final, and every copy has landed and been read)
    bool done = true;
    if (warp >= 1) done = mbar_wait(&accum, 0);
    tc_fence_after();
    if (!(ok && done)) set_status(a.status, GALE_ERR_TIMEOUT);
    const int quarter = warp & 3;
    const int64_t row = int64_t(rt) * kMxTile + quarter * 32 + lane;
    const uint32_t lanes = uint32_t(quarter) << 21;
    if (a.split == 1) {
        if (warp >= 2) {
            for (int c = 0; c < a.n; c += 16) {
                float v[16];
                tmem_ld16(tmem + lanes + c, v);
                if (row < a.rows) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (t0 + c + i < a.tokens) store_rn(a.y, a.ydtype, (t0 + c + i) * a.ldy + row, v[i]);
                }
            }
        }
    } else {
        // partial sums [token][128 rows] over the ring, which is no longer in use
        __syncthreads();
        float* ps = reinterpret_cast<float*>(smem);
        if (warp >= 2) {
            for (int c = 0; c < a.n; c += 16) {
                float v[16];
                tmem_ld16(tmem + lanes + c, v);
#pragma unroll
                for (int i = 0; i < 16; ++i) ps[(c + i) * kMxTile + quarter * 32 + lane] = v[i];
            }
        }
        cluster_sync();
        const int live = int(min(int64_t(a.n), a.tokens - t0)) * kMxTile;
        const uint32_t base = smem_u32(ps);
        for (int i = part * kGThreads + threadIdx.x; i < live; i += a.split * kGThreads) {
            float v = 0.f;
            for (int q = 0; q < a.split; ++q) v += ld_cluster_f32(base + i * 4, q);
            const int64_t r = int64_t(rt) * kMxTile + (i & (kMxTile - 1));
            if (r < a.rows) store_rn(a.y, a.ydtype, int64_t(t0 + i / kMxTile) * a.ldy + r, v);
        }
        cluster_sync();      // the peers have read this CTA's partial sums
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, a.cols);
}

// Tokens of a tile: all of them up to 256 (the MMA's N in steps of 16), equal
// tiles of a multiple of 64 beyond (a tile's first scale sits at an even TMEM column).
int gemm_tile_tokens(int64_t tokens) {
    if (tokens <= kGMaxN) return int(align_up(tokens, 16));
    const int64_t tiles = (tokens + kGMaxN - 1) / kGMaxN;
    return int(align_up((tokens + tiles - 1) / tiles, 64));
}

struct GemmPlan {
    GemmArgs a;
    int64_t grid;
    int smem;
};

void gemm_plan(int64_t rows, int nt, int64_t tokens, GemmPlan& p) {
    GemmArgs& a = p.a;
    a.rows = rows;
    a.tokens = tokens;
    a.nt = nt;
    a.n = gemm_tile_tokens(tokens);
    a.ntt = int((tokens + a.n - 1) / a.n);
    // tokens t0 .. t0 + n - 1 of a tile that starts at a multiple of n
    a.xatoms = a.ntt == 1 ? (a.n + kMxTile - 1) / kMxTile : a.n % kMxTile == 0 ? a.n / kMxTile : a.n / kMxTile + 2;
    if (a.xatoms > 3) a.xatoms = 3;
    const int64_t tiles = (rows + kMxTile - 1) / kMxTile * a.ntt;
    a.split = 1;
    if (a.n <= 64)
        while (a.split < 8 && tiles * a.split < 2 * sm_count() && nt / (a.split * 2) >= 4) a.split *= 2;
    a.stage_bytes = int(align_up(kGABytes + a.n * kMxTile + kMxAtomBytes * (1 + a.xatoms), 1024));
    // small tiles: two CTAs per SM, so that one's start and end overlap the other's stream
    const int room = (a.n <= 64 ? kGSmemSm / 2 : kGSmemSm) - 2048;
    a.stages = room / a.stage_bytes;
    if (a.stages > kGMaxStages) a.stages = kGMaxStages;
    int cols = 32;
    while (cols < a.n + a.stages * kGSfCols) cols *= 2;
    a.cols = cols;
    p.smem = a.stages * a.stage_bytes + 1024;
    // As large a share of the SM's shared memory as of its TMEM, so that a CTA
    // that is resident never waits for TMEM columns.
    const int least = int(int64_t(kGSmemSm) * cols / 512);
    if (p.smem < least) p.smem = least;
    p.grid = tiles * a.split;
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
    GemmPlan p{};
    gemm_plan(rows, int(W.cols_padded / kMxTile), tokens, p);
    if (p.grid > INT32_MAX) return GALE_ERR_UNSUPPORTED;
    p.a.wsc = w + W.s_offset;
    p.a.xsc = x + X.s_offset;
    p.a.y = y;
    p.a.status = static_cast<int32_t*>(ws);
    p.a.ldy = ldy;
    p.a.ydtype = y_dtype;
    CUtensorMap wmap, xmap;
    int rc = make_map_mx4(&wmap, w, W.q_bytes / (kMxTile / 2));
    if (rc == GALE_OK) rc = make_map_bytes(&xmap, x, W.cols_padded, tokens, kMxTile, p.a.n);
    if (rc != GALE_OK) return rc;
    if (ensure_smem(reinterpret_cast<const void*>(mx_gemm_kernel), p.smem) != GALE_OK) return GALE_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(p.grid));
    cfg.blockDim = dim3(kGThreads);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = as_stream(stream);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {unsigned(p.a.split), 1, 1};
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, mx_gemm_kernel, wmap, xmap, p.a) != cudaSuccess) {
        cudaGetLastError();      // reported here, not by the next call
        return GALE_ERR_CUDA;
    }
    return GALE_OK;
}
