// Softmax cross entropy over a vocabulary, and its backward pass, without the
// [M, V] logits.
//
//   l = x W^T            x [M,D], W [V,D]
//   lse_m = log sum_v exp(l_mv),  loss_m = lse_m - l_m,target(m)
//   dl_mv = g_m (exp(l_mv - lse_m) - [v = target(m)])
//   dx = dl W,  dW = dl^T x
//
// Forward: one product whose epilogue reduces each tile row to its maximum
// and its sum of exp(l - maximum) (8 bytes for 256 logits); a second kernel
// joins the tiles of a row.  Backward, piece by piece of the vocabulary: the
// piece's logits again, turned into dl in the epilogue and kept in 16 bits;
// then the piece's part of dx (summed over the pieces in fp32) and its rows
// of dW, all over the rows that are not ignored alone.  8 M V D flops in all, 2
// of them for the logits that were not kept.
//
// dl in 16 bits: |exp(l - lse) - [.]| <= 1, and a softmax over V entries is
// mostly values near 1/V, which fp16 holds with few bits or none.  So dl is kept
// as c_m K (exp(l - lse) - [.]) with K = 2^15 in fp16 (exact scaling; bf16
// needs none), c_m = g_m / max |g|, and max |g| / K is applied in fp32 to the
// sums.
#include "xent.h"

#include "layer_pipe.h"
#include "linear.h"

namespace pgemm {
namespace layer {
namespace {

template <class E>
constexpr float grad_scale() {
    return std::is_same<E, F16>::value ? 32768.0f : 1.0f;
}

// Rows of a tile to (maximum, sum of exponentials), and the target's logit
// from whichever lane holds it.  In registers, and with workgroups that walk
// the tiles: 8192 x 2048 x 65536 bf16 1575-1730 us (1270-1400 TFLOP/s); through LDS,
// one workgroup per tile, 1913.  Each row block's target is loaded where it is
// used: eight waits for memory a tile.
struct StatsEpi {
    static constexpr lp::EpiKind kind = lp::kRows;
    static constexpr bool kWalk = true;
    float2* part;  // [tile][M]
    float* target_logit;
    const int64_t* target;
    int64_t v0;     // vocabulary index of the product's column 0
    int64_t M;
    int columns;  // of the product
    int tile0;
    typedef float2 Acc;  // maximum, sum of exp(value - maximum)
    template <int FN>
    __device__ __forceinline__ Acc reduce(int r, bool valid, int col,
                                          const float (&v)[FN][4]) const {
        const int64_t t = valid ? target[r] - v0 - col : -1;  // in this lane: 16 j + q
        float m = -INFINITY;
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) m = fmaxf(m, v[j][q]);
        if (t >= 0 && t < 16 * FN && (t & 15) < 4 && t + col < columns) {
            float at = 0.0f;
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (t == 16 * j + q) at = v[j][q];
            target_logit[r] = at;
        }
        const float base = m == -INFINITY ? 0.0f : m;  // a row of -inf has the sum 0
        // exp(v - base) = exp2(v k - base k), k = log2 e; near the end of fp32's range
        // base k would overflow, and any k will do: what is not base is 0.
        const float k = fabsf(base) > 2e38f ? 1.0f : kLog2e;
        const float scaled = base * k;
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                s += __builtin_amdgcn_exp2f(fmaf(v[j][q], k, -scaled));
        return float2{m, s};
    }
    __device__ __forceinline__ void join(Acc& a, Acc b) const {
        const float m = fmaxf(a.x, b.x);
        const float base = m == -INFINITY ? 0.0f : m;
        a.y = a.y * exp_fast(a.x - base) + b.y * exp_fast(b.x - base);
        a.x = m;
    }
    __device__ __forceinline__ void finish(Acc a, int r, int tile) const {
        part[(int64_t)(tile0 + tile) * M + r] = a;
    }
};

// Joins a row's tiles: 16 rows per workgroup, 64 lanes taking every 64th tile
// of a row each (4 loads in flight), then the lanes in order through LDS; 8192
// rows of 256 tiles in 6 us (with 4 lanes a row 28).  A
// target outside the vocabulary that is not ignore_index gives NaN.
__global__ __launch_bounds__(1024) void join_kernel(const float2* __restrict__ part, int tiles,
                                                    const float* __restrict__ target_logit,
                                                    const int64_t* __restrict__ target,
                                                    int64_t ignore_index, int64_t V, int64_t M,
                                                    float* __restrict__ lse,
                                                    float* __restrict__ row_loss) {
    __shared__ float2 seg[64][16];
    const int row = threadIdx.x & 15, w = threadIdx.x >> 4;
    const int64_t r = (int64_t)blockIdx.x * 16 + row;
    float m = -INFINITY, s = 0.0f;
    auto join = [&](float2 p) {
        const float top = fmaxf(m, p.x);
        const float base = top == -INFINITY ? 0.0f : top;
        s = s * exp_fast(m - base) + p.y * exp_fast(p.x - base);
        m = top;
    };
    if (r < M) {
        int t = w;
        for (; t + 192 < tiles; t += 256) {
            float2 p[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) p[u] = part[(int64_t)(t + 64 * u) * M + r];
#pragma unroll
            for (int u = 0; u < 4; ++u) join(p[u]);
        }
        for (; t < tiles; t += 64) join(part[(int64_t)t * M + r]);
    }
    seg[w][row] = float2{m, s};
    for (int h = 32; h > 0; h >>= 1) {
        __syncthreads();
        if (w < h) {
            join(seg[w + h][row]);
            seg[w][row] = float2{m, s};
        }
    }
    if (w == 0 && r < M) {
        const float l = (m == -INFINITY ? 0.0f : m) + logf(s);
        lse[r] = l;
        const int64_t t = target[r];
        if (row_loss)
            row_loss[r] = t == ignore_index ? 0.0f
                          : (t >= 0 && t < V) ? l - target_logit[r]
                                              : __builtin_nanf("");
    }
}

// Sum (or mean over the rows that count) of the row losses, in fp64, by one
// workgroup in a fixed order.
__global__ __launch_bounds__(1024) void total_kernel(const float* __restrict__ row_loss,
                                                     const int64_t* __restrict__ target,
                                                     int64_t ignore_index, int64_t M, int mean,
                                                     float* __restrict__ loss) {
    __shared__ double sums[1024];
    __shared__ int64_t counts[1024];
    double s = 0.0;
    int64_t n = 0;
    for (int64_t r = threadIdx.x; r < M; r += 1024) {
        s += (double)row_loss[r];
        n += target[r] != ignore_index;
    }
    sums[threadIdx.x] = s;
    counts[threadIdx.x] = n;
    for (int h = 512; h > 0; h >>= 1) {
        __syncthreads();
        if (threadIdx.x < h) {
            sums[threadIdx.x] += sums[threadIdx.x + h];
            counts[threadIdx.x] += counts[threadIdx.x + h];
        }
    }
    if (threadIdx.x == 0) {
        const double d = mean ? (double)(counts[0] > 0 ? counts[0] : 1) : 1.0;
        loss[0] = (float)(sums[0] / d);
    }
}

// Row weights of the backward pass: c_m in [-1, 1], the factor of the sums,
// and the rows that count (c_m not 0) packed together, by one workgroup whose
// threads take consecutive runs of rows.  Ignored rows weigh 0; a weight that
// is not finite, or belongs to an invalid target (NaN), stands for its row
// alone.  Bound by latency: 8192 rows 25 us, of 4.5 ms that follow.
//   rank[m]: place of row m among the rows that count, -1 where it does not;
//   row[j]: the j-th row that counts; live: how many there are.
struct Kept {
    int* rank;
    int* row;
    int* live;
    float* weight;    // [j]
    float* lse;       // [j]
    int64_t* target;  // [j]
    float* factor;
};

__global__ __launch_bounds__(1024) void weights_kernel(const int64_t* __restrict__ target,
                                                       int64_t ignore_index, int64_t V, int64_t M,
                                                       int reduction,
                                                       const float* __restrict__ dloss,
                                                       const float* __restrict__ lse, float scale,
                                                       const Kept k) {
    __shared__ float tops[1024];
    __shared__ int counts[1024];
    __shared__ int places[1024];
    const int t = threadIdx.x;
    const bool each = reduction == PGEMM_REDUCE_NONE && dloss;
    const int64_t per = (M + 1023) / 1024;
    const int64_t r0 = t * per, r1 = r0 + per < M ? r0 + per : M;
    float top = 0.0f;
    int n = 0;
    for (int64_t r = r0; r < r1; ++r) {
        if (target[r] == ignore_index) continue;
        ++n;
        if (each) {
            const float a = fabsf(dloss[r]);
            if (a < INFINITY) top = fmaxf(top, a);
        }
    }
    tops[t] = top;
    counts[t] = n;
    for (int h = 512; h > 0; h >>= 1) {
        __syncthreads();
        if (t < h) {
            tops[t] = fmaxf(tops[t], tops[t + h]);
            counts[t] += counts[t + h];
        }
    }
    __syncthreads();
    top = tops[0];
    auto weight = [&](int64_t r) {
        const int64_t at = target[r];
        if (at == ignore_index) return 0.0f;
        if (at < 0 || at >= V) return __builtin_nanf("");
        if (!each) return 1.0f;
        const float g = dloss[r];
        return fabsf(g) < INFINITY ? (top > 0.0f ? g / top : 0.0f) : g;
    };
    int mine = 0;
    for (int64_t r = r0; r < r1; ++r) mine += weight(r) != 0.0f;
    places[t] = mine;
    for (int h = 1; h < 1024; h <<= 1) {  // running sums
        __syncthreads();
        const int before = t >= h ? places[t - h] : 0;
        __syncthreads();
        places[t] += before;
    }
    int j = places[t] - mine;
    for (int64_t r = r0; r < r1; ++r) {
        const float c = weight(r);
        k.rank[r] = c != 0.0f ? j : -1;
        if (c != 0.0f) {
            k.row[j] = (int)r;
            k.weight[j] = c;
            k.lse[j] = lse[r];
            k.target[j] = target[r];
            ++j;
        }
    }
    if (t == 1023) k.live[0] = places[1023];
    if (t == 0) {
        float f = each ? top : (dloss ? dloss[0] : 1.0f);
        if (reduction == PGEMM_REDUCE_MEAN) f /= (float)(counts[0] > 0 ? counts[0] : 1);
        k.factor[0] = f / scale;
    }
}

// The rows of x that count, packed together in padded rows of whole chunks;
// the rows of dx (where asked for) that do not are zeroed.  Bound by memory
// (8192 x 2048: 11.5 us for 63 MB, 5.5 TB/s).
__global__ __launch_bounds__(256) void gather_kernel(const Rows x, const Rows dx, uint16_t* kept,
                                                     int kept_ld, const int* __restrict__ rank,
                                                     int64_t M, int D) {
    const int cpr = (D + 7) / 8;
    const int64_t total = M * cpr;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / cpr;
        const int col = (int)(i - r * cpr) * 8, nv = min(8, D - col);
        const int j = rank[r];
        if (j >= 0) {
            *reinterpret_cast<u4_t*>(kept + (int64_t)j * kept_ld + col) =
                load8_bits(x.from(r), 0, col, nv);
        } else if (dx) {
            const float zero[8] = {};
            store8<F16, false>(dx.from(r), 0, col, nv, zero);
        }
    }
}

// dl of a piece: whole chunks, zeros past its last column.  7372 x 2048 x 32768
// bf16 780-810 us (1220-1270 TFLOP/s): an exponential and the weight a value, and
// 16 bits written.
template <class E>
struct DlogitEpi {
    static constexpr lp::EpiKind kind = lp::kPlain;
    static constexpr bool kWalk = false;
    static constexpr bool kRedo = false;
    static constexpr int kAhead = 8;
    Rows dl;
    const float* lse;
    const float* weight;
    const int64_t* target;
    int64_t v0;
    __device__ __forceinline__ DlogitEpi from(int64_t r) const {
        return {dl.from(r), lse + r, weight + r, target + r, v0};
    }
    struct Row {
        float weight, lse;
        int64_t target;
    };
    __device__ __forceinline__ bool aligned() const { return true; }
    template <bool STREAM, class Run>
    __device__ __forceinline__ void with(Run&& run) const {
        run(*this);
    }
    __device__ __forceinline__ lp::Nothing column(int, int) const { return {}; }
    __device__ __forceinline__ Row load(int row, int, int) const {
        return {weight[row], lse[row], target[row]};
    }
    __device__ __forceinline__ void operator()(int row, int col, int nv, float (&v)[8], lp::Nothing,
                                               const Row& aux) const {
        const float c = aux.weight * grad_scale<E>();
        const float l = aux.lse;
        const int64_t t = aux.target - v0 - col;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const float p = exp_fast(v[q] - l) - (t == q ? 1.0f : 0.0f);
            v[q] = q < nv ? c * p : 0.0f;
        }
        store8<E, true>(dl, row, col, 8, v);
    }
};

// The gradients' epilogue.  dx over the pieces: fp32 sums in the workspace, the
// last piece rounds; its rows go where the rows that count came from (map).  dx
// of a piece of 32768 at 7372 x 2048 675-710 us, its dW 717-746 (1330-1470 TFLOP/s).
template <class E>
struct SumEpi {
    static constexpr lp::EpiKind kind = lp::kPlain;
    static constexpr bool kWalk = false;
    static constexpr bool kRedo = false;
    static constexpr int kAhead = 4;
    float* sum;  // [M][ld], NULL where there is one piece only
    int ld;
    Rows out;
    const int* map;  // NULL: rows as they are
    const float* factor;
    int first, last;
    __device__ __forceinline__ SumEpi from(int64_t r) const {
        return {sum ? sum + r * ld : sum, ld,   map ? out : out.from(r), map ? map + r : map,
                factor,                   first, last};
    }
    struct Before {
        floatx4 lo, hi;
        int row;
    };
    __device__ __forceinline__ bool aligned() const { return out.aligned; }
    template <bool STREAM, class Run>
    __device__ __forceinline__ void with(Run&& run) const {
        run([this](int row, int col, int nv, float(&v)[8], float f, const Before& b)
                __attribute__((always_inline)) { put<STREAM>(row, col, nv, v, f, b); });
    }
    __device__ __forceinline__ float column(int, int) const { return factor[0]; }
    __device__ __forceinline__ Before load(int row, int col, int) const {
        Before b = {};
        if (map && last) b.row = map[row];
        if (!sum || first) return b;
        const float* p = sum + (uint32_t)(row * ld + col);
        b.lo = *reinterpret_cast<const floatx4*>(p);
        b.hi = *reinterpret_cast<const floatx4*>(p + 4);
        return b;
    }
    template <bool STREAM>
    __device__ __forceinline__ void put(int row, int col, int nv, float (&v)[8], float f,
                                        const Before& b) const {
        if (sum) {
            float* p = sum + (uint32_t)(row * ld + col);
            floatx4 lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
            if (!first) {
                lo += b.lo;
                hi += b.hi;
            }
            if (!last) {
                *reinterpret_cast<floatx4*>(p) = lo;
                *reinterpret_cast<floatx4*>(p + 4) = hi;
                return;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v[q] = lo[q];
                v[4 + q] = hi[q];
            }
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] *= f;
        if (map)
            store8<E, STREAM>(out.from(b.row), 0, col, nv, v);
        else
            store8<E, STREAM>(out, row, col, nv, v);
    }
};

// Vocabulary entries per piece: at most `most` bytes of dl, pieces of equal
// size and whole tiles.
constexpr int64_t kPieceBytes = (int64_t)1 << 29;
constexpr int64_t kPieceLeast = 1024;
constexpr int64_t kPieceMost = (int64_t)1 << 21;  // a row pitch of dl
constexpr int64_t kPackRows = 32768;  // rows of W padded at a time

int64_t piece_rows(int64_t V, int64_t most) {
    most = std::min(std::max(most / 256 * 256, kPieceLeast), kPieceMost);
    const int64_t n = (V + most - 1) / most;
    return n <= 1 ? V : round_up((V + n - 1) / n, 256);
}

// Rows v0 .. v0+n-1 of W as an operand, from where they lie or padded into `room`.
hipError_t piece(const void* w, int64_t ldw, int64_t v0, int64_t n, int64_t D, uint16_t* room,
                 bool dry, hipStream_t stream, View& out) {
    const uint16_t* p = static_cast<const uint16_t*>(w) + v0 * ldw;
    if (direct(w, ldw, D)) {
        out = {p, (int)ldw};
        return hipSuccess;
    }
    const int64_t d8 = round_up(D, 8);
    out = {room, (int)d8};
    return dry ? hipSuccess : launch_pack(p, ldw, room, d8, n, D, stream);
}

template <class E>
struct Xent {
    static hipError_t forward(const XentCall& c, Arena& ar, hipStream_t stream) {
        const int cus = compute_units();
        const bool straight = direct(c.w, c.ldw, c.D);
        const int64_t step = straight ? c.V : piece_rows(c.V, kPackRows);
        hipError_t rc;
        View x, w;
        if ((rc = operand(c.x, c.ldx, c.M, c.D, ar, stream, x)) != hipSuccess) return rc;
        uint16_t* room = nullptr;
        if (!straight) room = static_cast<uint16_t*>(ar.take(step * round_up(c.D, 8) * 2));
        const Cut cut = choose_cut(c.M, step, c.D, cus, 1);
        const int64_t bn = cut.big ? 256 : 128;
        const int64_t tiles = (c.V + step - 1) / step * ((step + bn - 1) / bn);
        float2* part = static_cast<float2*>(ar.take(tiles * c.M * 8));
        float* logit = static_cast<float*>(ar.take(c.M * 4));
        const bool total = c.reduction != PGEMM_REDUCE_NONE;
        float* row_loss = c.loss;
        if (total) row_loss = static_cast<float*>(ar.take(c.M * 4));
        if (ar.dry()) return hipSuccess;
        int used = 0;
        for (int64_t v0 = 0; c.M > 0 && v0 < c.V; v0 += step) {
            const int64_t n = std::min(step, c.V - v0);
            if ((rc = piece(c.w, c.ldw, v0, n, c.D, room, false, stream, w)) != hipSuccess)
                return rc;
            const Args g = args(x, w, c.M, n, c.D, cut, ar);
            const StatsEpi epi = {part, logit, c.target, v0, c.M, (int)n, used};
            using T = lp::Tiles<E, true, true>;
            rc = cut.big ? lp::launch_tiles<typename T::Big, StatsEpi, false>(g, 1, epi, stream)
                         : lp::launch_tiles<typename T::Small, StatsEpi, false>(g, 1, epi, stream);
            if (rc != hipSuccess) return rc;
            used += (int)((n + bn - 1) / bn);
        }
        if (c.M > 0) {
            hipLaunchKernelGGL(join_kernel, dim3((unsigned)((c.M + 15) / 16)), dim3(1024), 0, stream,
                               part, used, logit, c.target, c.ignore_index, c.V, c.M, c.lse,
                               row_loss);
            if ((rc = hipGetLastError()) != hipSuccess) return rc;
        }
        if (total) {
            hipLaunchKernelGGL(total_kernel, dim3(1), dim3(1024), 0, stream, row_loss, c.target,
                               c.ignore_index, c.M, (int)(c.reduction == PGEMM_REDUCE_MEAN), c.loss);
            return hipGetLastError();
        }
        return hipSuccess;
    }

    static hipError_t backward(const XentGradCall& c, Arena& ar, hipStream_t stream) {
        const int cus = compute_units();
        hipError_t rc;
        View w;
        const int64_t step = piece_rows(c.V, kPieceBytes / (2 * std::max<int64_t>(c.M, 1)));
        const int64_t s8 = round_up(step, 8), d8 = round_up(c.D, 8);
        const int64_t pieces = (c.V + step - 1) / step;
        uint16_t* room = nullptr;
        if (!direct(c.w, c.ldw, c.D)) room = static_cast<uint16_t*>(ar.take(step * d8 * 2));
        // The rows that count are packed together: the products take them
        // alone, and nothing of an ignored row (it may hold anything) reaches
        // a gradient.  The copy also serves as x in whole chunks.
        Kept k;
        k.rank = static_cast<int*>(ar.take(c.M * 4));
        k.row = static_cast<int*>(ar.take(c.M * 4));
        k.weight = static_cast<float*>(ar.take(c.M * 4));
        k.lse = static_cast<float*>(ar.take(c.M * 4));
        k.target = static_cast<int64_t*>(ar.take(c.M * 8));
        k.live = static_cast<int*>(ar.take(4));
        k.factor = static_cast<float*>(ar.take(4));
        uint16_t* kept = static_cast<uint16_t*>(ar.take(c.M * d8 * 2));
        uint16_t* dl = static_cast<uint16_t*>(ar.take(c.M * s8 * 2));
        float* sum = nullptr;
        if (c.dx && pieces > 1) sum = static_cast<float*>(ar.take(c.M * d8 * 4));
        // The three products of a piece share one buffer for their partials.
        const Cut cl = choose_cut(c.M, step, c.D, cus, 16), cx = choose_cut(c.M, c.D, step, cus, 16),
                  cw = choose_cut(step, c.D, c.M, cus, 16);
        const int64_t pb = std::max(part_bytes(cl, c.M, step),
                                    std::max(c.dx ? part_bytes(cx, c.M, c.D) : 0,
                                             c.dw ? part_bytes(cw, step, c.D) : 0));
        float* part = pb > 0 ? static_cast<float*>(ar.take(pb)) : nullptr;
        if (ar.dry()) return hipSuccess;
        auto product = [&](View a, View b, int64_t M, int64_t N, int64_t K) {
            Args g = {};
            g.a = a;
            g.b = b;
            g.M = (int)M;
            g.N = (int)N;
            g.K = (int)K;
            g.part = part;
            g.part_ld = (int)round_up(N, 8);
            g.live = k.live;
            return g;
        };
        hipLaunchKernelGGL(weights_kernel, dim3(1), dim3(1024), 0, stream, c.target, c.ignore_index,
                           c.V, c.M, c.reduction, c.dloss, c.lse, grad_scale<E>(), k);
        if ((rc = hipGetLastError()) != hipSuccess) return rc;
        if (c.M > 0 && c.D > 0) {
            const int64_t chunks = c.M * (d8 / 8);
            hipLaunchKernelGGL(gather_kernel,
                               dim3((unsigned)std::min<int64_t>((chunks + 255) / 256, 1 << 16)),
                               dim3(256), 0, stream, make_rows(c.x, c.ldx),
                               make_rows(c.dx, c.lddx), kept, (int)d8, k.rank, c.M, (int)c.D);
            if ((rc = hipGetLastError()) != hipSuccess) return rc;
        }
        const View x = {kept, (int)d8};
        for (int64_t v0 = 0; v0 < c.V; v0 += step) {
            const int64_t n = std::min(step, c.V - v0);
            const bool first = v0 == 0, last = v0 + n == c.V;
            if ((rc = piece(c.w, c.ldw, v0, n, c.D, room, false, stream, w)) != hipSuccess)
                return rc;
            const View dv = {dl, (int)s8};
            if (c.M > 0) {
                const DlogitEpi<E> epi = {{dl, (int)s8, 1}, k.lse, k.weight, k.target, v0};
                rc = lp::launch_product<E, true, true>(product(x, w, c.M, n, c.D), cl, epi, stream);
                if (rc != hipSuccess) return rc;
            }
            if (c.dx && c.M > 0 && c.D > 0) {
                const SumEpi<E> epi = {sum,      (int)d8, make_rows(c.dx, c.lddx), k.row,
                                       k.factor, first,   last};
                // the last piece may be shorter: its own contraction, the same cut
                Cut cut = cx;
                if (cut.splits > 1) cut.splits = (int)((n + cut.chunk - 1) / cut.chunk);
                rc = lp::launch_product<E, true, false>(product(dv, w, c.M, c.D, n), cut, epi,
                                                        stream);
                if (rc != hipSuccess) return rc;
            }
            if (c.dw && c.D > 0) {
                uint16_t* out = static_cast<uint16_t*>(c.dw) + v0 * c.lddw;
                const SumEpi<E> epi = {nullptr, 0, make_rows(out, c.lddw), nullptr, k.factor, 1, 1};
                rc = lp::launch_product<E, false, false>(product(dv, x, n, c.D, c.M), cw, epi,
                                                         stream);
                if (rc != hipSuccess) return rc;
            }
        }
        return hipSuccess;
    }
};

}  // namespace

hipError_t xent_forward(const XentCall& c, Arena& ar, hipStream_t stream) {
    return c.dtype == kBF16 ? Xent<BF16>::forward(c, ar, stream)
                            : Xent<F16>::forward(c, ar, stream);
}

hipError_t xent_backward(const XentGradCall& c, Arena& ar, hipStream_t stream) {
    return c.dtype == kBF16 ? Xent<BF16>::backward(c, ar, stream)
                            : Xent<F16>::backward(c, ar, stream);
}

}  // namespace layer
}  // namespace pgemm
