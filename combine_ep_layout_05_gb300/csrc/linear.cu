// Dense products with an epilogue (ep_linear) and the products of their
// gradients, for any number of rows.
//
//   out[r, c] = act(sum_l A(r, l) B(c, l) + bias[c]) + residual[r, c]
//
// bf16 operands, fp32 sums, one rounding at the end.  The tensor core cuts its
// sums off rather than rounding them, by about a unit in the last place for every 16 of the contraction: a sum of numbers of
// one sign lags behind by a share that grows with its length (measured: 2.6e-5 after 7168, 7.7e-5 after 16384, 3.3e-3
// after 2^19).  Up to kMostChain steps (8192) that is a fiftieth of the rounding to bf16, and bf16 results stay in
// tensor memory; longer contractions and all fp32 results are taken out every 512 and added in registers
// (LONG: 2e-6 off, however long; 2^17 takes 587 us instead of 574, 2^14 the same).  Three forms of the same
// loop, which differ in the way the operands lie in memory:
//   forward  A = x [M, K], B = w [N, K]: both along the contraction
//   grad_x   A = G [M, N], B = w [N, K]: B along its rows (columns of w)
//   grad_w   A = G [M, N], B = x [M, K]: both along their rows
// Nothing is transposed in memory: the tensor core reads either form from
// shared memory, with boxes of 128 rows (A's of as many as a tile has) x 64
// contraction or of 64 x 64.
//
// A CTA pair computes 256 x 256 outputs (SwiGLU: 256 x 128, the gate's rows in
// the first CTA's B, the up rows in the second's): each CTA holds 128 rows of A
// and 128 of B, 32 KB a step of 64, and its rows' accumulators.  A CTA alone
// (128 x 256) would write and read 96 KB of shared memory for each 512 cycles of
// products, a CTA of the pair 64.  Two accumulators of 256 columns alternate, so
// that one is stored while the other is summed.  Warps: 0 issues the boxes (whose
// bytes are counted on the first CTA's barrier, wherever they land), 1 the
// products (first CTA), 4 to 11 the epilogue: a thread owns a row of a half of
// the columns.
//
// Measured, from a graph: 8192 rows of 7168 -> 2 x 2048 with SwiGLU and pre-activations 258 us
// (1.87 PFLOP/s, 97% of the measured rate of library products; the tensor pipe is busy 87% of a cold launch), its two
// gradients 249 us each; 32768 rows of 7168 -> 256 in fp32 92 us (5.5 TB/s): in the first of two turns the memory
// bounds it, in the second the 32 KB a step that a CTA takes from L2 (0.27 us); their grad_x 100 us (470 MB written),
// bound by shared memory, through which operands, products and results go (some 1.6 us of a tile's 2.1).
#include <algorithm>

#include "linear_device.cuh"

namespace ep {

namespace {

constexpr int kThreads = 384;
constexpr int kRing = 192 * 1024;               // bytes of operands: 6 steps of whole tiles, at most kMostStages of less
constexpr int kMostStages = 16;
constexpr int kTile = 2 * kPart;                // rows and columns of a pair's tile
constexpr int kSegment = 8;                     // steps of a LONG sum that stay in tensor memory
constexpr int kIssueRegs = 88, kEndRegs = 208;  // LONG: 88 + 2 * 208 = 3 * 168, the launch's registers
constexpr int kGroup = 8;                       // row tiles that are walked together, for L2

struct LinearShared {
    unsigned char ring[kRing];                  // steps: A, then B
    unsigned char rows[8][32 * 128];            // a warp's results on their way out: 32 rows of 128 bytes
    uint64_t full[kMostStages];                 // (the first CTA's) both CTAs' operands
    uint64_t empty[kMostStages];                // a step's products are done
    uint64_t tfull[2];                          // an accumulator is complete
    uint64_t tempty[2];                         // (the first CTA's) taken out by both CTAs
    uint32_t tmem;
    int gave_up;
};

struct LinearMaps {
    CUtensorMap a, b, out;
};

// A unit of work: a tile and a part of the contraction
struct LinearUnit {
    int row, col, split, first, last;           // tile, part, steps [first, last)
};
__device__ __forceinline__ LinearUnit linear_unit(const LinearArgs &a, int u) {
    const int tiles = a.row_tiles * a.col_tiles;
    LinearUnit v;
    v.split = u / tiles;
    const int t = u - v.split * tiles, per = kGroup * a.col_tiles, g = t / per;
    const int in = t - g * per, n = min(kGroup, a.row_tiles - g * kGroup);
    v.row = g * kGroup + in % n;
    v.col = in / n;
    v.first = v.split * a.split_steps;
    v.last = min(v.first + a.split_steps, a.steps);
    return v;
}

// LONG: sums are taken out of tensor memory every kSegment steps and added in registers; OUT32: fp32 results (always
// LONG).
template <bool SWIGLU, bool A_MN, bool B_MN, bool LONG, bool OUT32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    linear_kernel(const __grid_constant__ LinearArgs a, const __grid_constant__ LinearMaps maps) {
    extern __shared__ __align__(1024) unsigned char raw[];    // (the only shared memory: it starts at its window's start)
    LinearShared &s = *reinterpret_cast<LinearShared *>(raw);
    // (gradients' tiles are whole)
    const int S = B_MN ? kRing / (2 * kPartBytes) : a.stages, stage_bytes = B_MN ? 2 * kPartBytes : a.stage_bytes;
    const int a_bytes = B_MN ? kPartBytes : a.a_bytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const int64_t all = (int64_t)a.row_tiles * a.col_tiles * a.splits;     // (below 2^31: checked on the host)
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int units = (int)all;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.tfull[i], 1);
            mbar_init(&s.tempty[i], 16);
        }
        s.gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<2>(&s.tmem);
    tmem_fence_before();
    __syncthreads();
    cluster_sync();    // the other CTA's barriers are there too
    tmem_fence_after();
    const uint32_t tmem = s.tmem;
    const Patience patience{&s.gave_up, a.wait_clocks};
    if (a.order == kAfter) wait_for_launch_before();
    let_next_launch_begin();

    if (LONG && warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (warp == 0) {
        // ---- boxes ----
        if (lane == 0) {
            const uint32_t full = cluster_addr(&s.full[0], 0);
            // (rows of A that a tile lacks stay whatever they are: they reach no other row's sums, and nobody takes theirs)
            const int bytes = 2 * (kStep * 2) * ((B_MN ? kPart : a.half_rows) + (B_MN ? kPart : a.half_cols));
            int st = 0, ph = 1, it = 0;
            bool ok = true;
            for (int u = pair; u < units && ok; u += pairs) {
                const LinearUnit v = linear_unit(a, u);
                const int r0 = (v.row * 2 + rank) * (B_MN ? kPart : a.half_rows);
                const int c0 = SWIGLU ? rank * (int)a.C + v.col * kPart : v.col * kTile + rank * (B_MN ? kPart : a.half_cols);
                for (int k = v.first; k < v.last; ++k, ++it) {
                    ok = mbar_wait(&s.empty[st], ph, patience);
                    if (!ok) break;
                    if (rank == 0) mbar_expect_tx(&s.full[st], bytes);
                    unsigned char *pa = s.ring + st * stage_bytes;
                    const uint32_t bar = full + st * 8;
                    if (A_MN) {
                        tma_load_2d_pair(pa, &maps.a, r0 * 2, k * kStep, bar);
                        tma_load_2d_pair(pa + kPartBytes / 2, &maps.a, r0 * 2 + 128, k * kStep, bar);
                    } else {
                        tma_load_2d_pair(pa, &maps.a, k * kStep * 2, r0, bar);
                    }
                    unsigned char *pb = pa + a_bytes;
                    if (B_MN) {
                        tma_load_2d_pair(pb, &maps.b, c0 * 2, k * kStep, bar);
                        tma_load_2d_pair(pb + kPartBytes / 2, &maps.b, c0 * 2 + 128, k * kStep, bar);
                    } else {
                        tma_load_2d_pair(pb, &maps.b, k * kStep * 2, c0, bar);
                    }
                    if (++st == S) { st = 0; ph ^= 1; }
                }
            }
            // the products of a step follow its boxes
            drain(s.empty, S, it);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---- products (the loop is the whole warp's, so that its values are uniform; one lane issues) ----
        if (rank == 0) {
            const uint32_t idesc = mma_idesc_bf16(kTile, B_MN ? kTile : 2 * a.half_cols, A_MN, B_MN);
            const bool issue = elect_one();
            const uint64_t da0 = A_MN ? smem_desc_mn(s.ring, kPartBytes / 2) : smem_desc(s.ring);
            const uint64_t db0 = B_MN ? smem_desc_mn(s.ring + a_bytes, kPartBytes / 2) : smem_desc(s.ring + a_bytes);
            // 16 of the contraction: 32 bytes along a row, or 16 lines of 128 bytes
            constexpr uint32_t ka = A_MN ? 2048 >> 4 : 32 >> 4, kb = B_MN ? 2048 >> 4 : 32 >> 4;
            int st = 0, ph = 0, acc = 0, aph = 1;
            bool ok = true;
            for (int u = pair; u < units && ok; u += pairs) {
                const LinearUnit v = linear_unit(a, u);
                for (int k0 = v.first; k0 < v.last && ok;) {
                    const int k1 = LONG ? min(k0 + kSegment, v.last) : v.last;
                    ok = warp_wait<true>(&s.tempty[acc], aph, patience);
                    if (!ok) break;
                    tmem_fence_after();
                    for (int k = k0; k < k1; ++k) {
                        ok = warp_wait<true>(&s.full[st], ph, patience);
                        if (!ok) break;
                        acquire_shared_of_cluster();
                        tmem_fence_after();
                        if (issue) {
                            const uint32_t at = (uint32_t)(st * (stage_bytes >> 4));
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                mma_bf16<2>(tmem + acc * kTile, da0 + at + i * ka, db0 + at + i * kb, idesc,
                                            k > k0 || i > 0);
                            mma_commit<2>(&s.empty[st]);
                        }
                        if (++st == S) { st = 0; ph ^= 1; }
                    }
                    if (!ok) break;
                    if (issue) mma_commit<2>(&s.tfull[acc]);
                    acc ^= 1;
                    aph ^= acc == 0;
                    k0 = k1;
                }
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        if (LONG) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEndRegs));
        // ---- epilogue (a gradient's products have nothing to add: PLAIN) ----
        constexpr bool PLAIN = A_MN || B_MN;
        const int half = (warp - 4) >> 2, quarter = warp & 3;
        constexpr int kCols = SWIGLU ? kPart / 2 : kPart;          // output columns of a thread
        constexpr int kChunks = kCols / 32, kWide = SWIGLU ? 64 : 32;
        const uint32_t tm = tmem + (uint32_t)(quarter * 32) * 65536 + half * kCols;
        const uint32_t tempty = cluster_addr(&s.tempty[0], 0);
        int acc = 0, ph = 0;
        // 32 columns of an accumulator (SwiGLU: of the gate, then of the up rows), started and waited for
        const auto start = [&](int q, uint32_t (&t)[kWide]) {
            const uint32_t at = tm + acc * kTile + q * 32;
            tmem_ld16(at, t);
            tmem_ld16(at + 16, t + 16);
            if (SWIGLU) {
                tmem_ld16(at + kPart, t + kWide - 32);
                tmem_ld16(at + kPart + 16, t + kWide - 16);
            }
        };
        const auto load = [&](int q, uint32_t (&t)[kWide]) {
            start(q, t);
            tmem_wait_ld<kWide>(t);
        };
        const auto taken_out = [&]() {
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_relaxed_cluster(tempty + acc * 8);
        };
        bool ok = true;
        for (int u = pair; u < units && ok; u += pairs) {
            const LinearUnit v = linear_unit(a, u);
            const int held = B_MN ? kPart : a.half_rows;
            const int64_t first = ((int64_t)v.row * 2 + rank) * held, r = first + quarter * 32 + lane;
            const int64_t end = min(a.R, first + held);
            const int64_t c0 = (int64_t)v.col * (SWIGLU ? kPart : kTile) + half * kCols;
            // the residual of 32 columns: where rows are aligned, asked for one step ahead of them
            uint32_t res[16];
            const auto ask = [&](int q) {
                if (PLAIN) return;
                const int64_t c = c0 + q * 32;
                const int n = (int)min(a.C - c, (int64_t)32);
                if (a.residual && a.residual_align >= 16 && r < end && n > 0)
                    load_bf16<32>(a.residual + r * a.residual_stride + c, res, n, a.residual_align);
            };
            ask(0);
            const int64_t row0 = r - lane;                      // the warp's rows, and how many exist
            const int n_rows = (int)min(max(end - row0, (int64_t)0), (int64_t)32);
            // Results leave through shared memory, in boxes of 32 rows x 128 bytes, where out can be a tensor map (each thread
            // storing 32 bytes a time along its row, a warp's store touches 32 lines: 32768 x 7168 of 256 took 115 us, 4.1
            // TB/s).  The swizzle keeps rows' 16 bytes apart.
            unsigned char *own = s.rows[warp - 4];
            const bool boxed = a.boxes && (n_rows == 32 || end == a.R);   // (a box of fewer rows would reach into the next tile)
            constexpr int kHalves = OUT32 ? 1 : 2;              // chunks of 32 columns in a box
            const auto finish = [&](int q, const uint32_t *t) {
                const int64_t c = c0 + q * 32;
                const int n = (int)min(a.C - c, (int64_t)32);
                if (n <= 0) return;                             // (for the whole warp)
                const bool live = r < end;
                if (boxed && q % kHalves == 0) {
                    if (lane == 0) bulk_wait_read<0>();       // (what was in this box has been read)
                    __syncwarp();
                }
                float z[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) z[i] = __uint_as_float(t[i]);
                if (!PLAIN) {
                    // bf16 pre-activations, as far as they are wanted
                    const auto keep = [&](const float(&v)[32], int64_t at) {
                        if (!a.pre) return;
                        if (a.pre_align >= 16) {
                            if (live) store_bf16(a.pre + r * a.pre_stride + at, v, n, a.pre_align);
                        } else {
                            put_row(own, v);
                            copy_out(own, a.pre + row0 * a.pre_stride + at, a.pre_stride, n_rows, n);
                        }
                    };
                    if (a.bias) add_vector(a.bias + c, z, n);
                    keep(z, c);
                    if (SWIGLU) {
                        float up[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) up[i] = __uint_as_float(t[kWide - 32 + i]);
                        if (a.bias) add_vector(a.bias + a.C + c, up, n);
                        keep(up, a.C + c);
#pragma unroll
                        for (int i = 0; i < 32; ++i) z[i] = swiglu(z[i], up[i]);
                    } else {
                        activate(z, a.act);
                    }
                    if (a.residual) {
                        if (a.residual_align < 16)
                            copy_in(own, a.residual + row0 * a.residual_stride + c, a.residual_stride, n_rows, n, res);
                        if (live) add_bf16<32>(res, z);
                        if (q + 1 < kChunks) ask(q + 1);
                    }
                }
                if (boxed) {
                    uint4 *to = reinterpret_cast<uint4 *>(own + lane * 128);
#pragma unroll
                    for (int i = 0; i < (OUT32 ? 8 : 4); ++i) {
                        const int at = (OUT32 ? i : q % kHalves * 4 + i) ^ (lane & 7);
                        if (OUT32)
                            to[at] = make_uint4(__float_as_uint(z[4 * i]), __float_as_uint(z[4 * i + 1]),
                                                __float_as_uint(z[4 * i + 2]), __float_as_uint(z[4 * i + 3]));
                        else
                            to[at] = make_uint4(pack_bf16x2(z[8 * i % 32], z[(8 * i + 1) % 32]),
                                                pack_bf16x2(z[(8 * i + 2) % 32], z[(8 * i + 3) % 32]),
                                                pack_bf16x2(z[(8 * i + 4) % 32], z[(8 * i + 5) % 32]),
                                                pack_bf16x2(z[(8 * i + 6) % 32], z[(8 * i + 7) % 32]));
                    }
                    if (q % kHalves == kHalves - 1 || a.C - c <= 32) {
                        fence_async_shared();
                        __syncwarp();
                        if (lane == 0 && n_rows > 0) {
                            tma_store_3d(&maps.out, (int)(c - q % kHalves * 32) * (OUT32 ? 4 : 2), (int)row0, v.split, own);
                            bulk_commit();
                        }
                    }
                } else if (OUT32) {
                    float *out = reinterpret_cast<float *>(a.out) + v.split * a.split_stride;
                    if (a.out_align >= 16) {
                        if (live) store_fp32(out + r * a.out_stride + c, z, n, a.out_align);
                    } else {
                        put_row_fp32(own, z);
                        copy_out_fp32(own, out + row0 * a.out_stride + c, a.out_stride, n_rows, n);
                    }
                } else {
                    uint16_t *out = reinterpret_cast<uint16_t *>(a.out);
                    if (a.out_align >= 16) {
                        if (live) store_bf16(out + r * a.out_stride + c, z, n, a.out_align);
                    } else {
                        put_row(own, z);
                        copy_out(own, out + row0 * a.out_stride + c, a.out_stride, n_rows, n);
                    }
                }
            };
            if (LONG) {
                float sum[kChunks][kWide];
#pragma unroll
                for (int q = 0; q < kChunks; ++q)
#pragma unroll
                    for (int i = 0; i < kWide; ++i) sum[q][i] = 0.f;
                for (int k = v.first; k < v.last; k += kSegment) {
                    ok = warp_wait(&s.tfull[acc], ph, patience);
                    if (!ok) break;
                    tmem_fence_after();
#pragma unroll
                    for (int q = 0; q < kChunks; ++q) {
                        uint32_t t[kWide];
                        load(q, t);
#pragma unroll
                        for (int i = 0; i < kWide; ++i) sum[q][i] += __uint_as_float(t[i]);
                    }
                    taken_out();
                    acc ^= 1;
                    ph ^= acc == 0;
                }
                if (!ok) break;
#pragma unroll
                for (int q = 0; q < kChunks; ++q) finish(q, reinterpret_cast<const uint32_t *>(sum[q]));
            } else {
                ok = warp_wait(&s.tfull[acc], ph, patience);
                if (!ok) break;
                tmem_fence_after();
#pragma unroll 1
                for (int q = 0; q < kChunks; ++q) {
                    __syncwarp();              // (lanes whose rows do not exist come back early)
                    uint32_t t[kWide];
                    load(q, t);
                    if (q == kChunks - 1) taken_out();
                    finish(q, t);
                }
                acc ^= 1;
                ph ^= acc == 0;
            }
            __syncwarp();
        }
        if (a.boxes && lane == 0) bulk_wait_all();
    }
    tmem_fence_before();
    __syncthreads();
    cluster_sync();    // nothing arrives here any more, and what reads this CTA's shared memory is done
    if (warp == 1) {
        tmem_fence_after();
        tmem_free<2>(tmem);
    }
    if (threadIdx.x == 0 && s.gave_up) raise_status(a.dev_status, EP_STATUS_TIMEOUT);
    if (a.order == kBeside) wait_for_launch_before();
}

// The operand as a tensor map of bytes.  Along the contraction: boxes of `rows`
// rows x 128 bytes; along its rows: boxes of 64 of the contraction x 128 bytes.
cudaError_t operand_map(const LinearOperand &o, bool mn, int rows, CUtensorMap *map) {
    const cuuint64_t dims[2] = {(cuuint64_t)o.cols * 2, (cuuint64_t)o.rows}, strides[1] = {(cuuint64_t)o.stride * 2};
    const cuuint32_t box[2] = {128, (cuuint32_t)(mn ? kStep : rows)};
    return encode_map(map, 2, o.p, dims, strides, box);
}

template <bool SWIGLU, bool A_MN, bool B_MN, bool LONG, bool OUT32>
cudaError_t launch(const LinearArgs &a, const LinearMaps &maps, cudaStream_t st) {
    constexpr int bytes = sizeof(LinearShared);
    static_assert(bytes <= 227 * 1024, "shared memory");
    static std::atomic<int> ready[kCacheDevices];
    cudaError_t e = cudaSuccess;
    cached_per_device(ready, [&](int) {
        e = cudaFuncSetAttribute(linear_kernel<SWIGLU, A_MN, B_MN, LONG, OUT32>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        // the warpgroups' register shares are drawn from what the block was launched with
        cudaFuncAttributes f{};
        if (!e) e = cudaFuncGetAttributes(&f, linear_kernel<SWIGLU, A_MN, B_MN, LONG, OUT32>);
        if (!e && LONG && f.numRegs * 3 < kIssueRegs + 2 * kEndRegs) e = cudaErrorInvalidDeviceFunction;
        return e == cudaSuccess ? 1 : 0;
    });
    if (e) return e;
    const int64_t units = (int64_t)a.row_tiles * a.col_tiles * a.splits;
    const int grid = (int)std::min<int64_t>(num_sms() & ~1, 2 * units);
    return launch_in_order(a.order, linear_kernel<SWIGLU, A_MN, B_MN, LONG, OUT32>, dim3(grid), kThreads, bytes, 0, st, a, maps);
}

// the same, by how results are summed
template <bool SWIGLU, bool A_MN, bool B_MN>
cudaError_t launch_sums(const LinearArgs &a, bool longer, const LinearMaps &maps, cudaStream_t st) {
    if (a.out32) return launch<SWIGLU, A_MN, B_MN, true, true>(a, maps, st);
    return longer ? launch<SWIGLU, A_MN, B_MN, true, false>(a, maps, st) : launch<SWIGLU, A_MN, B_MN, false, false>(a, maps, st);
}

}  // namespace

// What a launch of this kernel takes, in us, fitted to measurements from a graph: 28 tiles of 4, 16, 32 and 112 steps
// 7.1, 11.1, 15.4 and 36.8 us; 84 tiles of 32 steps 25.0; 3584 of 4 steps 106 (there the epilogue is what takes the
// time, 2.2 us a tile).  A split contraction adds the parts' sum: their bytes at 5 TB/s and a launch.
// The shorter of this and linear_few_time() says which kernel a call takes.  Each forced, in us (few rows' kernel |
// this one), forward, bf16 results: 7168 -> 256 at 16, 512, 4096 rows 7.1 | 35, 10.6 | 36, 20.6 | 36; 7168 -> 2048 with SwiGLU
// at 1, 512, 1024, 4096 rows 11.2 | 36, 31.7 | 37, 54 | 38, 207 | 137; 2048 -> 7168 at 128, 256, 512 rows 11.8 | 14.9, 15.1 |
// 15.0, 22.2 | 15.6.  fp32 results: 7168 -> 256 at 16, 512, 2048 rows 7.1 | 36, 10.6 | 36, 15.6 | 37; where the few rows' kernel
// would have to keep more than kChain steps in an accumulator, this one takes the call although it is slower: 4096 rows 25 |
// 37 (from 2433 rows on), 256 rows of the SwiGLU 24 | 37, 2048 of 1024 -> 1024 13.5 | 15.9.  grad_x of 2048 -> 1024 at 515 and
// 2048 rows 10.8 | 9.9, 17.3 | 10.3; grad_w 10.6 | 9.3, 17.0 | 15.7.
double linear_time(int64_t R, int64_t C, int64_t L, bool swiglu, int splits) {
    const int64_t cols = swiglu ? kPart : kTile, tiles = ((R + kTile - 1) / kTile) * ((C + cols - 1) / cols);
    const int64_t steps = ((L + kStep - 1) / kStep + splits - 1) / splits, turns = (tiles * splits + 75) / 76;
    return 6.8 + 0.27 * steps + (turns - 1) * std::max(0.27 * steps + 1.0, 2.2) +
           (splits > 1 ? 3.0 + 4e-6 * R * C * (splits + 1) / 5.0 : 0.0);
}

int linear_splits(int64_t R, int64_t C, int64_t L) {
    const int64_t steps = (L + kStep - 1) / kStep;
    int best = 1;
    double least = 1e30;
    for (int s = 1; s <= std::min<int64_t>(steps, 16); ++s) {
        const int64_t per = (steps + s - 1) / s;
        if ((steps + per - 1) / per != s) continue;          // every part has steps
        const double t = linear_time(R, C, L, false, s);
        if (t < least) { least = t; best = s; }
    }
    return best;
}

cudaError_t launch_linear(int form, LinearArgs a, const LinearOperand &A, const LinearOperand &B, cudaStream_t st) {
    const bool swiglu = form == kFormForward && a.act == EP_ACT_SWIGLU;
    const int cols = swiglu ? kPart : kTile;
    a.col_tiles = (int)((a.C + cols - 1) / cols);
    a.steps = (int)((a.L + kStep - 1) / kStep);
    a.split_steps = (a.steps + a.splits - 1) / a.splits;
    a.half_rows = a.half_cols = kPart;
    // One tile of columns: A is read from memory once, and bounds the launch.  (1) The columns are as many as there are, which
    // leaves room for more steps under way: 6000 and 20000 rows of 7168 -> 64, cold, in us, whole tiles | as many as there
    // are: 41 | 37, 74 | 68.  (2) Where whole tiles would leave half of the SMs or more without work in the last turn, the turns
    // are made equal in rows.  A turn of products takes as long, but the memory has the same work all the time.  Cold,
    // 7168 -> 256, whole | equal: 20000 rows (the last turn has 3 of 76 pairs) 98 | 84, 28000 (34) 100 | 94, 44000 (20)
    // 146 | 136, 65536 (28) 192 | 187; 32768 (52) 98.1 | 103.9.  A single turn is not cut: its 112 steps take as long either way.
    if (form == kFormForward && a.col_tiles == 1) {
        if (!swiglu) a.half_cols = (int)(std::max<int64_t>(a.C, 32) + 15) / 16 * 8;
        const int64_t pairs = num_sms() / 2, tiles = (a.R + kTile - 1) / kTile, turns = (tiles + pairs - 1) / pairs;
        if (turns > 1 && (tiles - (turns - 1) * pairs) * 2 <= pairs)
            a.half_rows = (int)((a.R + 2 * turns * pairs - 1) / (2 * turns * pairs));
    }
    a.row_tiles = (int)((a.R + 2 * a.half_rows - 1) / (2 * a.half_rows));
    // (parts start at whole atoms of 8 rows)
    a.a_bytes = (a.half_rows + 7) / 8 * 8 * kStep * 2;
    a.stage_bytes = a.a_bytes + a.half_cols * kStep * 2;
    a.stages = std::min(kMostStages, kRing / a.stage_bytes);
    LinearMaps maps;
    if (cudaError_t e = operand_map(A, form == kFormGradW, a.half_rows, &maps.a)) return e;
    if (cudaError_t e = operand_map(B, form != kFormForward, a.half_cols, &maps.b)) return e;
    // (rows and their strides in multiples of 16 bytes; the parts of a split contraction are its third dimension)
    const int64_t size = a.out32 ? 4 : 2, stride = a.out_stride * size, part = (a.splits > 1 ? a.split_stride : a.out_stride) * size;
    // (not where the pre-activations or the residual need that memory)
    a.boxes = a.out_align >= 16 && a.C * size % 16 == 0 && stride < (int64_t)1 << 40 && part < (int64_t)1 << 40 &&
              !(a.pre && a.pre_align < 16) && !(a.residual && a.residual_align < 16);
    maps.out = maps.a;
    if (a.boxes) {
        const cuuint64_t dims[3] = {(cuuint64_t)(a.C * size), (cuuint64_t)a.R, (cuuint64_t)a.splits};
        const cuuint64_t strides[2] = {(cuuint64_t)stride, (cuuint64_t)part};
        const cuuint32_t box[3] = {128, 32, 1};
        if (cudaError_t e = encode_map(&maps.out, 3, a.out, dims, strides, box)) return e;
    }
    const bool longer = a.split_steps > kMostChain;
    if (form == kFormGradX) return launch_sums<false, false, true>(a, longer, maps, st);
    if (form == kFormGradW) return launch_sums<false, true, true>(a, longer, maps, st);
    return swiglu ? launch_sums<true, false, false>(a, longer, maps, st) : launch_sums<false, false, false>(a, longer, maps, st);
}

}  // namespace ep
