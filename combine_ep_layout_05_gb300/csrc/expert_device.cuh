// What both expert kernels share: the work list over experts, row tiles and
// column tiles, and the receive rows of an expert.
#pragma once

#include "tcgen05.cuh"

namespace ep {

namespace {

constexpr int kBlock = 128;                     // channels, and matrix rows, of a scale
constexpr int kOperand = kBlock * kBlock;       // bytes of 128 rows x 128 channels

// Experts' rows and the row tiles before each expert
struct WorkList {
    int first[kMaxExperts + 1];
    int rows[kMaxExperts];
};

// Fills the list for tiles of tile_rows rows; called by all threads of the
// block (threads a multiple of 32), the list is complete when it returns.
__device__ __forceinline__ void make_list(WorkList &s, const ExpertArgs &a, int tile_rows, int threads) {
    const Dims &d = a.d;
    const int E = (int)d.E, lane = threadIdx.x & 31;
    bool bad = false;
    for (int e = threadIdx.x; e < E; e += threads) {
        int n = 0;
        for (int r = 0; r < d.R; ++r) {
            const int c = a.tokens_per_expert[(int64_t)r * E + e];
            const int ok = min(max(c, 0), (int)d.Tr);
            bad |= ok != c;
            n += ok;
        }
        s.rows[e] = n;
    }
    if (bad && blockIdx.x == 0) raise_status(a.dev_status, EP_STATUS_BAD_SLOT);
    __syncthreads();
    if (threadIdx.x < 32) {
        int sum = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int t = e0 + lane < E ? (s.rows[e0 + lane] + tile_rows - 1) / tile_rows : 0;
            int inc = t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(kFull, inc, o);
                if (lane >= o) inc += v;
            }
            if (e0 + lane < E) s.first[e0 + lane] = sum + inc - t;
            sum += __shfl_sync(kFull, inc, 31);
        }
        if (lane == 0) s.first[E] = sum;
    }
    __syncthreads();
}

// One unit of work
struct Unit {
    int e, m0;        // expert and its first row
    int rows;         // rows from m0 on (at most the tile's)
    int nb;           // column tile
};

__device__ __forceinline__ Unit find_unit(const WorkList &s, int E, int tile_rows, int col_tiles, int u) {
    // the last e with first[e] * col_tiles <= u (experts without rows share their successor's first tile)
    int lo = 0, hi = E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s.first[mid] * col_tiles <= u) lo = mid;
        else hi = mid;
    }
    const int tiles = s.first[lo + 1] - s.first[lo];
    const int r = u - s.first[lo] * col_tiles;
    Unit v;
    v.e = lo;
    v.nb = r / tiles;                 // row tiles fastest: they share the matrix rows
    v.m0 = (r % tiles) * tile_rows;
    v.rows = min(tile_rows, s.rows[lo] - v.m0);
    return v;
}

// Receive rows of rows m[] of expert e, for each lane (called by whole warps;
// counts outside [0, Tr] are clamped).
template <int N>
__device__ __forceinline__ void receive_rows(const ExpertArgs &a, int e, const int (&m)[N], int (&row)[N]) {
    const Dims &d = a.d;
    const int lane = threadIdx.x & 31, R = (int)d.R, Tr = (int)d.Tr;
#pragma unroll
    for (int i = 0; i < N; ++i) row[i] = e * R * Tr + m[i];
    int before = 0;
    for (int r0 = 0; r0 < R; r0 += 32) {
        const int r = r0 + lane;
        int end = r < R ? min(max(a.tokens_per_expert[(int64_t)r * d.E + e], 0), Tr) : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFull, end, o);
            if (lane >= o) end += v;
        }
        end += before;                // rows up to and with source r
        const int last = min(32, R - r0);
        for (int i = 0; i < last; ++i) {
            const int to = __shfl_sync(kFull, end, i);
            const int start = (e * R + r0 + i + 1) * Tr - to;   // of the next source's segment, less the rows before
#pragma unroll
            for (int x = 0; x < N; ++x)
                if (to <= m[x]) row[x] = start + m[x];
        }
        before = __shfl_sync(kFull, end, 31);
    }
}

// the matrices as a tensor map of bytes: boxes of box_rows rows x 128 channels
inline cudaError_t matrix_map(const ExpertArgs &a, int box_rows, CUtensorMap *map) {
    const cuuint64_t dims[3] = {(cuuint64_t)a.K, (cuuint64_t)a.N, (cuuint64_t)a.d.E};
    const cuuint64_t strides[2] = {(cuuint64_t)a.K, (cuuint64_t)(a.N * a.K)};
    const cuuint32_t box[3] = {kBlock, (cuuint32_t)box_rows, 1};
    return encode_map(map, 3, a.w, dims, strides, box);
}

}  // namespace

}  // namespace ep
