// Dense products with an epilogue for few rows, and their gradients where tiles are few:
// the matrix is read once, and that is what takes the time.
//
// Same operation as linear.cu, in the same three forms, with the operands' parts
// exchanged: 128 columns of the output are the tensor core's M (forward: 128 rows of the
// matrix; SwiGLU: 64 gate and 64 up rows), its rows the N (16, 32, .. 128).
// A tile of 128 matrix rows alone would leave most SMs idle (a gate of 256 experts has
// two), so the CTAs of a cluster share a tile's contraction: each sums its part in
// tensor memory, puts it into its shared memory, and then finishes a share of
// the tile's outputs, whose parts it reads from the shared memory of every CTA of the
// cluster, in the order of their ranks.  No workspace, no atomics, one order of the sums.
// Two CTAs to an SM, so that one streams while the other starts or ends.
//
// The tensor core cuts its sums off rather than rounding them (linear.cu).  Every kChain steps go to an
// accumulator of their own, and these are added in fp32.  Where accumulators do not suffice, an
// accumulator takes more, at most kMostChain, for a bf16 result; for an fp32 result, or for longer ones, the
// other kernel does the work.
//
// Measured, from a graph, operands in L2: 32 rows of 7168 -> 256 (a gate) 7.0 us, of which the launch, the tensor memory, the
// first boxes and the exchange take 5; 512 rows 10.6 us; one row of 7168 -> 2 x 2048 with SwiGLU 11.2 us.  Where the
// SwiGLU's matrix comes from memory, as in a decode step, it takes 17.2 us (59 MB, 3.4 TB/s).
#include <algorithm>
#include <cstddef>

#include "linear_device.cuh"

namespace ep {

namespace {

constexpr int kThreads = 256;                   // warp 0: boxes, 1: products; all: the end
constexpr int kMaxStages = 6;
constexpr int kRing = 112 * 1024;               // bytes of operands: two CTAs an SM
constexpr int kColumns = 256;                   // of tensor memory, likewise
constexpr int kChain = 8;                       // steps in one accumulator, if accumulators suffice

struct FewBarriers {
    uint64_t full[kMaxStages], empty[kMaxStages], summed;
    uint32_t tmem;
    int gave_up;
};

struct FewMaps {
    CUtensorMap r, c;        // the operands of the rows, and of the columns
};

// How a launch is cut
struct FewPlan {
    int col_tiles, tile_rows;    // rows of x in a tile
    int rows;                // the same up to a multiple of 16, in a box
    int stage, stages;       // bytes of a step's operands, buffers
    int steps, split_steps;  // of the contraction, and at most of a CTA
    int chain, accs;         // steps of an accumulator, accumulators
};

// 4 numbers of the shared memory of a CTA of the cluster
__device__ __forceinline__ float4 load_cluster(uint32_t addr) {
    float4 x;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                 : "r"(addr)
                 : "memory");
    return x;
}
// v += N CTAs' numbers at `at`, from rank q on, loads first
template <int N>
__device__ __forceinline__ void add_parts(float (&v)[4], const float *at, uint32_t q) {
    float4 x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = load_cluster(cluster_addr(at, q + i));
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[0] += x[i].x;
        v[1] += x[i].y;
        v[2] += x[i].z;
        v[3] += x[i].w;
    }
}
// the same of all CTAs (a power of two of them)
__device__ __forceinline__ void add_all(float (&v)[4], const float *at, uint32_t size) {
    if (size >= 8)
        for (uint32_t q = 0; q < size; q += 8) add_parts<8>(v, at, q);
    else if (size == 4) add_parts<4>(v, at, 0);
    else if (size == 2) add_parts<2>(v, at, 0);
    else add_parts<1>(v, at, 0);
}
// 4 consecutive bf16 of a row, of which n exist; vec: 8-byte accesses are aligned
__device__ __forceinline__ void store4(uint16_t *p, const float (&v)[4], int n, bool vec) {
    const uint32_t lo = pack_bf16x2(v[0], v[1]), hi = pack_bf16x2(v[2], v[3]);
    if (vec && n >= 4) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(lo, hi);
    } else {
        p[0] = (uint16_t)lo;
        if (n > 1) p[1] = (uint16_t)(lo >> 16);
        if (n > 2) p[2] = (uint16_t)hi;
        if (n > 3) p[3] = (uint16_t)(hi >> 16);
    }
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

// R_MN, C_MN: operands along their rows, as in linear.cu (A_MN and B_MN there)
template <bool SWIGLU, bool R_MN, bool C_MN>
__global__ void __launch_bounds__(kThreads, 2)
    linear_few_kernel(const __grid_constant__ LinearArgs a, const __grid_constant__ FewMaps maps, const FewPlan p) {
    extern __shared__ __align__(1024) unsigned char raw[];    // (the only shared memory: it starts at its window's start)
    FewBarriers &s = *reinterpret_cast<FewBarriers *>(raw + p.stage * p.stages);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank(), size = cluster_size();
    // the tile: column tiles of a row tile follow one another
    const int tile = blockIdx.x / size, col = tile % p.col_tiles;
    const int64_t row0 = (int64_t)(tile / p.col_tiles) * p.tile_rows;
    const int rows = (int)min((int64_t)p.tile_rows, a.R - row0);
    const int first = min((int)rank * p.split_steps, p.steps), last = min(first + p.split_steps, p.steps);

    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        mbar_init(&s.summed, 1);
        s.gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s.tmem)),
                     "n"(kColumns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = s.tmem;
    const Patience patience{&s.gave_up, a.wait_clocks};
    if (a.order == kAfter) wait_for_launch_before();
    let_next_launch_begin();

    if (warp == 0) {
        if (lane == 0) {
            // the tile's two halves of 64 columns
            const int c0 = col * (SWIGLU ? kPart / 2 : kPart), c1 = SWIGLU ? (int)a.C + c0 : c0 + kPart / 2;
            int st = 0, ph = 1, it = 0;
            for (int k = first; k < last; ++k, ++it) {
                if (!mbar_wait(&s.empty[st], ph, patience)) break;
                mbar_expect_tx(&s.full[st], p.stage);
                unsigned char *buf = raw + st * p.stage;
                tma_load_2d(buf, &maps.c, C_MN ? c0 * 2 : k * kStep * 2, C_MN ? k * kStep : c0, &s.full[st]);
                tma_load_2d(buf + kPartBytes / 2, &maps.c, C_MN ? c1 * 2 : k * kStep * 2, C_MN ? k * kStep : c1,
                            &s.full[st]);
                buf += kPartBytes;
                if (R_MN)
                    for (int i = 0; i < p.rows; i += 64)
                        tma_load_2d(buf + i * 128, &maps.r, (int)row0 * 2 + i * 2, k * kStep, &s.full[st]);
                else
                    tma_load_2d(buf, &maps.r, k * kStep * 2, (int)row0, &s.full[st]);
                if (++st == p.stages) { st = 0; ph ^= 1; }
            }
            // what has been issued lands, whether its products were or not (together within a second)
            const long long t0 = clock64();
            for (int i = max(0, it - p.stages); i < it; ++i)
                while (!mbar_try_wait(&s.full[i % p.stages], i / p.stages & 1))
                    if (clock64() - t0 > (1ll << 31)) break;
        }
        __syncwarp();
    } else if (warp == 1) {
        const bool issue = elect_one();
        const uint32_t idesc = mma_idesc_bf16(kPart, p.rows, C_MN, R_MN);
        const uint64_t dc = C_MN ? smem_desc_mn(raw, kPartBytes / 2) : smem_desc(raw);
        const uint64_t dr = R_MN ? smem_desc_mn(raw + kPartBytes, kPartBytes / 2) : smem_desc(raw + kPartBytes);
        // 16 of the contraction: 32 bytes along a row, or 16 lines of 128 bytes
        constexpr uint32_t kc = C_MN ? 2048 >> 4 : 32 >> 4, kr = R_MN ? 2048 >> 4 : 32 >> 4;
        int st = 0, ph = 0;
        bool ok = true;
        for (int k = first; k < last; ++k) {
            ok = warp_wait(&s.full[st], ph, patience);
            if (!ok) break;
            tmem_fence_after();
            if (issue) {
                const uint32_t buf = (uint32_t)(st * p.stage >> 4);
                const int at = k - first, acc = at / p.chain;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mma_bf16<1>(tmem + acc * p.rows, dc + buf + i * kc, dr + buf + i * kr, idesc, at % p.chain > 0 || i > 0);
                mma_commit<1>(&s.empty[st]);
            }
            if (++st == p.stages) { st = 0; ph ^= 1; }
        }
        if (issue) mma_commit<1>(&s.summed);      // (of all that were issued, given up or not)
        __syncwarp();
    }
    // ---- this CTA's part of the sums -> shared memory, [row of x][matrix row]; the operands are done with ----
    __syncwarp();
    float *part = reinterpret_cast<float *>(raw);
    if (!warp_wait(&s.summed, 0, patience)) {
        const long long t0 = clock64();            // (issued products end by themselves)
        while (!mbar_try_wait(&s.summed, 0))
            if (clock64() - t0 > (1ll << 31)) break;
        __syncwarp();
    }
    tmem_fence_after();
    __syncthreads();                               // (the boxes have landed, too)
    {
        const int quarter = warp & 3, half = warp >> 2, mine = quarter * 32 + lane;
        const int accs = (last - first + p.chain - 1) / p.chain;
        for (int c = half * 16; c < p.rows; c += 32) {
            float v[16] = {};
            for (int i = 0; i < accs; ++i) {
                uint32_t t[16];
                tmem_ld16(tmem + (uint32_t)(quarter * 32) * 65536 + i * p.rows + c, t);
                tmem_wait_ld<16>(t);
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] += __uint_as_float(t[j]);
            }
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (c + j < rows) part[(c + j) * kPart + mine] = v[j];
        }
    }
    tmem_fence_before();
    __syncthreads();
    cluster_sync();
    // ---- a share of the outputs, 4 columns a turn ----
    {
        constexpr int W = (SWIGLU ? kPart / 2 : kPart) / 4;
        const int items = rows * W, share = (items + (int)size - 1) / (int)size;
        const int end = min(items, (int)(rank + 1) * share);
        for (int i = (int)rank * share + threadIdx.x; i < end; i += kThreads) {
            const int r = i / W, at = i % W * 4;
            const int64_t m = row0 + r, c = (int64_t)col * (W * 4) + at;
            const int n = (int)min(a.C - c, (int64_t)4);
            if (n <= 0) continue;
            float z[4] = {}, up[4] = {};
            add_all(z, &part[r * kPart + at], size);
            if (SWIGLU) add_all(up, &part[r * kPart + W * 4 + at], size);
            if (a.bias) add_vector(a.bias + c, z, n);
            if (SWIGLU && a.bias) add_vector(a.bias + a.C + c, up, n);
            if (a.pre) {
                uint16_t *pre = a.pre + m * a.pre_stride + c;
                store4(pre, z, n, a.pre_align >= 16);
                if (SWIGLU) store4(pre + a.C, up, n, a.pre_align >= 16);
            }
            if (SWIGLU) {
#pragma unroll
                for (int j = 0; j < 4; ++j) z[j] = swiglu(z[j], up[j]);
            } else {
                activate(z, a.act);
            }
            if (a.residual) {
                const uint16_t *res = a.residual + m * a.residual_stride + c;
                if (n >= 4 && a.residual_align >= 16) {
                    const uint2 v = *reinterpret_cast<const uint2 *>(res);
                    z[0] += bf16_lo(v.x);
                    z[1] += bf16_hi(v.x);
                    z[2] += bf16_lo(v.y);
                    z[3] += bf16_hi(v.y);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < n) z[j] += __uint_as_float((uint32_t)res[j] << 16);
                }
            }
            if (a.out32) {
                float *out = reinterpret_cast<float *>(a.out) + m * a.out_stride + c;
                if (n >= 4 && a.out_align >= 16) {
                    *reinterpret_cast<float4 *>(out) = make_float4(z[0], z[1], z[2], z[3]);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < n) out[j] = z[j];
                }
            } else {
                store4(reinterpret_cast<uint16_t *>(a.out) + m * a.out_stride + c, z, n, a.out_align >= 16);
            }
        }
    }
    __syncwarp();                                  // (lanes leave that loop at different turns; the barrier is the whole warp's)
    cluster_sync();                                // nobody reads this CTA's part any more
    if (warp == 1) {
        tmem_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kColumns));
    }
    if (threadIdx.x == 0 && s.gave_up) raise_status(a.dev_status, EP_STATUS_TIMEOUT);
    if (a.order == kBeside) wait_for_launch_before();
}

template <bool SWIGLU, bool R_MN, bool C_MN>
cudaError_t launch(const LinearArgs &a, const FewMaps &maps, const FewPlan &p, int tiles, int size, cudaStream_t st) {
    static std::atomic<int> ready[kCacheDevices];
    cudaError_t e = cudaSuccess;
    cached_per_device(ready, [&](int) {
        e = cudaFuncSetAttribute(linear_few_kernel<SWIGLU, R_MN, C_MN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kRing + (int)sizeof(FewBarriers));
        if (!e) e = cudaFuncSetAttribute(linear_few_kernel<SWIGLU, R_MN, C_MN>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        return e == cudaSuccess ? 1 : 0;
    });
    if (e) return e;
    return launch_in_order(a.order, linear_few_kernel<SWIGLU, R_MN, C_MN>, dim3((unsigned)(tiles * size)), kThreads,
                           p.stage * p.stages + sizeof(FewBarriers), size, st, a, maps, p);
}

}  // namespace

namespace {

// How few rows are cut, and by how many CTAs to a tile.
//
// The CTAs of a cluster take, in us (measured from a graph, fitted to 16 to 128 rows of a tile, 2 to 112 steps and 1 to
// 16 CTAs to a tile): each step 0.24 and 0.002 a row, little more where two CTAs share an SM, but not less than the memory;
// the exchange of the parts 0.0015 a row and CTA of the cluster; each CTA 0.006 to start, and 5 in all, which every turn of
// the SMs costs again (32768 x 7168 of 64: 458 us here, 47 turns; some 105 by the other kernel).  Clusters of 16 find their places slowly: 128 of their
// CTAs took 13.2 us for what 64 CTAs of clusters of 8 did in 11.9, 64 of them 10.4 against 11.7.
FewPlan few_plan(int form, const LinearArgs &a, int &size, int64_t &tiles, double &time) {
    const bool swiglu = a.act == EP_ACT_SWIGLU;
    FewPlan best;
    FewPlan p;
    // (fp32 results: half the rows, for twice the accumulators)
    const int most = a.out32 ? kPart / 2 : kPart, outs = swiglu ? kPart / 2 : kPart;
    const int64_t row_tiles = (a.R + most - 1) / most;
    // (tiles of equal rows; but boxes of an operand along its rows have to start at multiples of 16 bytes, so these tiles are
    // whole boxes of 64 rows)
    p.tile_rows = (int)(row_tiles > 1 && form == kFormGradW ? most : (a.R + row_tiles - 1) / row_tiles);
    p.rows = (p.tile_rows + 15) / 16 * 16;
    // (an operand along its rows comes in boxes of 64 of them)
    p.stage = kPartBytes + (form == kFormGradW ? (p.rows + 63) / 64 * 64 : p.rows) * kStep * 2;
    p.stages = std::min(kMaxStages, kRing / p.stage);
    p.steps = (int)((a.L + kStep - 1) / kStep);
    p.col_tiles = (int)((a.C + outs - 1) / outs);
    tiles = row_tiles * p.col_tiles;
    time = 1e30;
    for (int c = 1; c <= 16; c *= 2) {
        const int64_t ctas = tiles * c;
        if (c > 1 && (c > p.steps || ctas > (c == 16 ? 64 : 304))) break;
        p.split_steps = (p.steps + c - 1) / c;
        p.accs = std::min(kColumns / p.rows, (p.split_steps + kChain - 1) / kChain);
        p.chain = (p.split_steps + p.accs - 1) / p.accs;
        const double turns = (double)((ctas + 303) / 304);
        const double step = (0.24 + 0.002 * p.rows) * (ctas > 152 ? 1.05 : 1.0);
        const double bytes = 2.0 * a.L * (outs * (swiglu ? 2 : 1)) * p.col_tiles;
        const double start = 5.0 + 0.006 * std::min<int64_t>(ctas, 304) + 0.0015 * c * p.rows;
        double t = turns * start + std::max(turns * step * p.split_steps, bytes / 6.8e6);
        // a longer chain would cost the result digits
        if (p.chain > (a.out32 ? kChain : kMostChain)) t += 1e9;
        if (t < time) {
            time = t;
            best = p;
            size = c;
        }
    }
    return best;
}

}  // namespace

double linear_few_time(int form, const LinearArgs &a) {
    int size;
    int64_t tiles;
    double time;
    few_plan(form, a, size, tiles, time);
    return time;
}

cudaError_t launch_linear_few(int form, const LinearArgs &a, const LinearOperand &A, const LinearOperand &B,
                              cudaStream_t st) {
    int size;
    int64_t tiles;
    double time;
    const FewPlan p = few_plan(form, a, size, tiles, time);
    if (tiles * size >= (int64_t)1 << 31) return cudaErrorInvalidConfiguration;    // (a self-test; otherwise the other kernel's)
    const bool r_mn = form == kFormGradW, c_mn = form != kFormForward;
    FewMaps maps;
    const auto map = [](const LinearOperand &o, int rows, CUtensorMap *m) {
        const cuuint64_t dims[2] = {(cuuint64_t)o.cols * 2, (cuuint64_t)o.rows}, strides[1] = {(cuuint64_t)o.stride * 2};
        const cuuint32_t box[2] = {128, (cuuint32_t)rows};
        return encode_map(m, 2, o.p, dims, strides, box);
    };
    if (cudaError_t e = map(A, r_mn ? kStep : p.rows, &maps.r)) return e;
    if (cudaError_t e = map(B, c_mn ? kStep : kPart / 2, &maps.c)) return e;
    if (form == kFormGradX) return launch<false, false, true>(a, maps, p, (int)tiles, size, st);
    if (form == kFormGradW) return launch<false, true, true>(a, maps, p, (int)tiles, size, st);
    return a.act == EP_ACT_SWIGLU ? launch<true, false, false>(a, maps, p, (int)tiles, size, st)
                                  : launch<false, false, false>(a, maps, p, (int)tiles, size, st);
}

}  // namespace ep
