// The layer norm's backward pass. With hat = (z - mean) * rstd and d = dy * weight,
//
//   dx      = R(rstd * (d - sum d / H - hat * sum(d * hat) / H) + dz)
//   dweight = sum over the rows of dy * hat
//   dbias   = sum over the rows of dy
//
// where DDP_RMS_NORM has no mean and no sum d / H. One pass over memory, bound by
// it: a row stays in registers between its two sums and dx, and each thread
// keeps the sums of its columns over all rows that its workgroup takes. Every
// workgroup leaves one row of such sums (a part), which a second launch adds
// up: no atomics, and an order that the sizes and types decide. 32768 rows of 2048
// bf16 values take 87 us and the join 4 (5.8 TB/s together), 2048 rows of 1024 fp32
// values 6 to 9 and 2 to 3.5.
#include "layernorm_kernels.h"

namespace ddp {
namespace {

// hat and d of one vector, zero in the columns that are skipped.
template <int X, int Y, int VEC>
__device__ __forceinline__ void normalise(const typename Raw<X, VEC>::type &z, const typename Raw<Y, VEC>::type &dy,
                                          float mean, float rstd, int skip, float (&hat)[VEC], float (&g)[VEC])
{
    widen_all<X, VEC>(z, hat);
    widen_all<Y, VEC>(dy, g);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        hat[j] = j >= skip ? (hat[j] - mean) * rstd : 0.0f;
        g[j] = j >= skip ? g[j] : 0.0f;
    }
}

// The sums that a row's dx takes off.
struct Along {
    float shift, slope;
    __device__ __forceinline__ Along(float d, float d_hat, const LayerArgs &a)
    {
        const float h = float(a.width);
        shift = a.rms ? 0.0f : d / h;
        slope = d_hat / h;
    }
};

template <int X, int VEC>
__device__ __forceinline__ void dx_of(const Along &k, float rstd, const float (&d)[VEC], const float (&hat)[VEC],
                                      const typename Raw<X, VEC>::type &dz, float (&v)[VEC])
{
    widen_all<X, VEC>(dz, v);
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = (d[j] - k.shift - hat[j] * k.slope) * rstd + v[j];
}

// Makes the compiler take a value for a new one: what was computed from it is
// computed again, where it would otherwise fill registers until then.
template <class V>
__device__ __forceinline__ void forget(V &x)
{
    if constexpr (sizeof(V) >= 8) {
        typedef uint32_t words __attribute__((ext_vector_type(sizeof(V) / 4)));
        words w = __builtin_bit_cast(words, x);
        asm volatile("" : "+v"(w));
        x = __builtin_bit_cast(V, w);
    }
}

// What R rows' backward pass reads, U vectors a thread.
template <int X, int Y, int T, int U, int R, int VEC>
struct Rows {
    typename Raw<X, VEC>::type z[R][U], dz[R][U];
    typename Raw<Y, VEC>::type dy[R][U];
    float mean[R], rstd[R];

    template <bool STREAM>
    __device__ __forceinline__ void load_as(const LayerArgs &a, const LayerBackward &b, int64_t row0, int t)
    {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = min(row0 + r, a.rows - 1);   // past the last row: the last again, not counted
            mean[r] = b.mean ? ((const GLOBAL float *)b.mean)[row] : 0.0f;
            rstd[r] = ((const GLOBAL float *)b.rstd)[row];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const Columns<VEC> c(u * T + t, a.width);
                z[r][u] = load<X, VEC, STREAM>(row_of<X>(b.z, row, a.z_stride), c.col);
                dy[r][u] = load<Y, VEC, STREAM>(row_of<Y>(b.dy, row, a.y_stride), c.col);
                dz[r][u] = 0;
                if (b.dz) dz[r][u] = load<X, VEC, STREAM>(row_of<X>(b.dz, row, a.z_stride), c.col);
            }
        }
    }
    __device__ __forceinline__ void load_rows(const LayerArgs &a, const LayerBackward &b, int64_t row0, int t)
    {
        if (a.stream)
            load_as<true>(a, b, row0, t);
        else
            load_as<false>(a, b, row0, t);
    }
};

// R rows at a time in the registers of T threads, U vectors of each: all their
// loads are under way before the first is used, those of the next rows too with
// AHEAD, and one barrier serves R rows. Between the sums and dx a row is kept as
// it was read. 32768 rows of 2048 bf16 values: one row at a time 111 us, two 103,
// four 107; two, read past the caches, 93, and with the next two ahead 91.
template <int X, int Y, int THREADS, int T, int U, int R, bool AHEAD, int VEC>
__global__ void __launch_bounds__(THREADS) layernorm_grad_rows(LayerArgs a, LayerBackward b)
{
    constexpr int GROUPS = THREADS / T;
    const int group = group_of<T>(), t = int(threadIdx.x) % T;
    float w[U][VEC], dw[U][VEC] = {}, db[U][VEC] = {};
#pragma unroll
    for (int u = 0; u < U; ++u)
        load_weight<VEC>(b.weight, a.weight_dtype, Columns<VEC>(u * T + t, a.width).col, 1.0f, w[u]);
    int turn = 0;
    const int64_t step = int64_t(b.n_parts) * GROUPS * R;
    Rows<X, Y, T, U, R, VEC> now, next;
    if (AHEAD) next.load_rows(a, b, (int64_t(blockIdx.x) * GROUPS + group) * R, t);
    // the same turns for all threads
    for (int64_t first = int64_t(blockIdx.x) * GROUPS * R; first < a.rows; first += step) {
        const int64_t row0 = first + group * R;
        if (AHEAD) {
            now = next;
            if (first + step < a.rows) next.load_rows(a, b, row0 + step, t);
        } else {
            now.load_rows(a, b, row0, t);
        }
        auto &[z, dz, dy, mean, rstd] = now;
        float s[2 * R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            s[2 * r] = s[2 * r + 1] = 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const Columns<VEC> c(u * T + t, a.width);
                float hat[VEC], g[VEC];
                normalise<X, Y, VEC>(z[r][u], dy[r][u], mean[r], rstd[r], row0 + r < a.rows ? c.skip : VEC, hat, g);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    dw[u][j] = __fmaf_rn(g[j], hat[j], dw[u][j]);
                    db[u][j] += g[j];
                    const float d = g[j] * w[u][j];
                    s[2 * r] += d;
                    s[2 * r + 1] = __fmaf_rn(d, hat[j], s[2 * r + 1]);
                }
            }
        }
        if (!b.dx) continue;
        row_sum<T, THREADS>(s, turn);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (row0 + r >= a.rows) continue;
            const Along k(s[2 * r], s[2 * r + 1], a);
            void *dx = row_of<X>(b.dx, row0 + r, a.x_stride);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const Columns<VEC> c(u * T + t, a.width);
                float hat[VEC], d[VEC], v[VEC];
                forget(z[r][u]);
                forget(dy[r][u]);
                normalise<X, Y, VEC>(z[r][u], dy[r][u], mean[r], rstd[r], c.skip, hat, d);
#pragma unroll
                for (int j = 0; j < VEC; ++j) d[j] *= w[u][j];
                dx_of<X, VEC>(k, rstd[r], d, hat, dz[r][u], v);
                if (c.skip < VEC) store<X, VEC>(dx, c.col, v, c.skip);
            }
        }
    }
    if (!b.parts) return;
    float *part = b.parts + int64_t(blockIdx.x) * 2 * a.width;
    if constexpr (GROUPS > 1) {
        // the groups' sums, added in order
        __shared__ float sums[2][GROUPS][T * VEC];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u > 0) __syncthreads();
#pragma unroll
            for (int j = 0; j < VEC; ++j) sums[0][group][t * VEC + j] = dw[u][j], sums[1][group][t * VEC + j] = db[u][j];
            __syncthreads();
            for (int i = int(threadIdx.x); i < (b.dbias ? 2 : 1) * T * VEC; i += THREADS) {
                const int which = i / (T * VEC), at = i % (T * VEC);
                const Columns<VEC> c(u * T + at / VEC, a.width);
                float v = sums[which][0][at];
#pragma unroll
                for (int k = 1; k < GROUPS; ++k) v += sums[which][k][at];
                if (at % VEC >= c.skip) ((GLOBAL float *)part)[which * a.width + c.col + at % VEC] = v;
            }
        }
    } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const Columns<VEC> c(u * T + t, a.width);
            if (c.skip < VEC) {
                store<DDP_F32, VEC>(part, c.col, dw[u], c.skip);
                if (b.dbias) store<DDP_F32, VEC>(part + a.width, c.col, db[u], c.skip);
            }
        }
    }
}

// dx of a row of any width by a workgroup, read twice. dx may lie where dy or
// dz does: a thread uses only columns that it writes itself.
template <int X, int Y, int VEC>
__global__ void __launch_bounds__(1024) layernorm_grad_wide(LayerArgs a, LayerBackward b, int64_t first)
{
    constexpr int T = 1024;
    const int64_t row = first + blockIdx.x;
    const void *z = row_of<X>(b.z, row, a.z_stride), *dy = row_of<Y>(b.dy, row, a.y_stride);
    void *dx = row_of<X>(b.dx, row, a.x_stride);
    const float mean = b.mean ? ((const GLOBAL float *)b.mean)[row] : 0.0f;
    const float rstd = ((const GLOBAL float *)b.rstd)[row];
    const int64_t vectors = (a.width + VEC - 1) / VEC;
    float hat[VEC], d[VEC];
    const auto take = [&](const Columns<VEC> &c) {
        float w[VEC];
        normalise<X, Y, VEC>(load<X, VEC>(z, c.col), load<Y, VEC>(dy, c.col), mean, rstd, c.skip, hat, d);
        load_weight<VEC>(b.weight, a.weight_dtype, c.col, 1.0f, w);
#pragma unroll
        for (int j = 0; j < VEC; ++j) d[j] *= w[j];
    };
    double sum = 0.0, along = 0.0;   // may be long
    for (int64_t i = threadIdx.x; i < vectors; i += T) {
        take(Columns<VEC>(i, a.width));
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            sum += double(d[j]);
            along = __fma_rn(double(d[j]), double(hat[j]), along);
        }
    }
    float s[2] = {float(sum), float(along)};
    int turn = 0;
    row_sum<T, T>(s, turn);
    const Along k(s[0], s[1], a);
    for (int64_t i = threadIdx.x; i < vectors; i += T) {
        const Columns<VEC> c(i, a.width);
        take(c);
        typename Raw<X, VEC>::type dz = 0;
        if (b.dz) dz = load<X, VEC>(row_of<X>(b.dz, row, a.z_stride), c.col);
        float v[VEC];
        dx_of<X, VEC>(k, rstd, d, hat, dz, v);
        store<X, VEC>(dx, c.col, v, c.skip);
    }
}

// The parts of rows of any width: a slab of 64 vectors of columns a workgroup,
// four rows at a time.
template <int X, int Y, int VEC>
__global__ void __launch_bounds__(256) layernorm_grad_columns(LayerArgs a, LayerBackward b)
{
    constexpr int GROUPS = 4;
    __shared__ float sums[2][GROUPS][64][VEC];
    const int group = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / 64), t = int(threadIdx.x) % 64;
    const Columns<VEC> c(int64_t(blockIdx.x) * 64 + t, a.width);
    float dw[VEC] = {}, db[VEC] = {};
    for (int64_t row = int64_t(blockIdx.y) * GROUPS + group; row < a.rows; row += int64_t(b.n_parts) * GROUPS) {
        const float mean = b.mean ? ((const GLOBAL float *)b.mean)[row] : 0.0f;
        const float rstd = ((const GLOBAL float *)b.rstd)[row];
        float hat[VEC], g[VEC];
        normalise<X, Y, VEC>(load<X, VEC>(row_of<X>(b.z, row, a.z_stride), c.col),
                             load<Y, VEC>(row_of<Y>(b.dy, row, a.y_stride), c.col), mean, rstd, c.skip, hat, g);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            dw[j] = __fmaf_rn(g[j], hat[j], dw[j]);
            db[j] += g[j];
        }
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) sums[0][group][t][j] = dw[j], sums[1][group][t][j] = db[j];
    __syncthreads();
    if (group < 2 && c.skip < VEC) {
        float v[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            v[j] = sums[group][0][t][j];
#pragma unroll
            for (int k = 1; k < GROUPS; ++k) v[j] += sums[group][k][t][j];
        }
        store<DDP_F32, VEC>(b.parts + (int64_t(blockIdx.y) * 2 + group) * a.width, c.col, v, c.skip);
    }
}

// One value of dweight or dbias, rounded once.
__device__ __forceinline__ void put_gradient(const LayerArgs &a, const LayerBackward &b, void *out, int64_t col, float v)
{
    const auto put = [&](auto type) {
        typedef Raw<decltype(type)::value, 1> R;
        GLOBAL typename R::elem *p = (GLOBAL typename R::elem *)out + col;
        *p = narrow<decltype(type)::value>(b.accumulate ? widen<decltype(type)::value>(*p) + v : v);
    };
    if (a.grad_dtype == DDP_F32)
        put(std::integral_constant<int, DDP_F32>());
    else if (a.grad_dtype == DDP_BF16)
        put(std::integral_constant<int, DDP_BF16>());
    else
        put(std::integral_constant<int, DDP_F16>());
}

// Sums of the parts, 32 columns a workgroup, each column's parts dealt to 32
// threads that add theirs in order, and then their sums.
constexpr int kJoinColumns = 32, kJoinSlices = 32;

__global__ void __launch_bounds__(kJoinColumns *kJoinSlices) layernorm_grad_join(LayerArgs a, LayerBackward b)
{
    __shared__ float sums[kJoinSlices][kJoinColumns];
    const int which = int(blockIdx.y), x = int(threadIdx.x) % kJoinColumns, slice = int(threadIdx.x) / kJoinColumns;
    void *out = which ? b.dbias : b.dweight;
    if (!out) return;
    const int64_t col = int64_t(blockIdx.x) * kJoinColumns + x;
    float s = 0.0f;
    if (col < a.width) {
        const GLOBAL float *p = (const GLOBAL float *)b.parts + which * a.width + col;
#pragma unroll 8
        for (int k = slice; k < b.n_parts; k += kJoinSlices) s += p[int64_t(k) * 2 * a.width];
    }
    sums[slice][x] = s;
    __syncthreads();
    if (slice > 0 || col >= a.width) return;
    s = sums[0][x];
#pragma unroll
    for (int k = 1; k < kJoinSlices; ++k) s += sums[k][x];
    put_gradient(a, b, out, col, s);
}

// A small call in one launch: the first workgroups take the weight's and bias's
// columns, the others the rows' dx. Both read z and dy, which the caches hold; it
// spares the parts and the launch that adds them (when it pays is the host's
// rule). dx may not lie where dy does.
constexpr int kSmallThreads = 512;
constexpr int kSlab = 4;   // vectors of columns of a workgroup: its threads go 128 rows at a time

// The sum over a wave's lanes that are alike modulo 4, in its first four.
__device__ __forceinline__ float over_slab(float x)
{
    x = with_lane<0x124>(x);   // four lanes on, of sixteen
    x = with_lane<0x128>(x);   // eight on
    return across_rows<64>(x);
}

// 32 columns' or so gradients over all rows, as the type that they have.
template <int X, int Y, int VEC>
__device__ __forceinline__ void small_columns(const LayerArgs &a, const LayerBackward &b)
{
    constexpr int GROUPS = kSmallThreads / kSlab, AHEAD = 4;
    __shared__ float sums[kSmallThreads / 64][kSlab][2 * VEC];
    const int lane = int(threadIdx.x) % kSlab, group = int(threadIdx.x) / kSlab;
    const Columns<VEC> c(int64_t(blockIdx.x) * kSlab + lane, a.width);
    float s[2 * VEC] = {};
    for (int64_t first = group; first < a.rows; first += AHEAD * GROUPS) {
        typename Raw<X, VEC>::type z[AHEAD];
        typename Raw<Y, VEC>::type dy[AHEAD];
        float mean[AHEAD], rstd[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int64_t row = min(first + k * GROUPS, a.rows - 1);   // past the last row: the last again, not counted
            mean[k] = b.mean ? ((const GLOBAL float *)b.mean)[row] : 0.0f;
            rstd[k] = ((const GLOBAL float *)b.rstd)[row];
            z[k] = load<X, VEC>(row_of<X>(b.z, row, a.z_stride), c.col);
            dy[k] = load<Y, VEC>(row_of<Y>(b.dy, row, a.y_stride), c.col);
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            float hat[VEC], g[VEC];
            normalise<X, Y, VEC>(z[k], dy[k], mean[k], rstd[k], first + k * GROUPS < a.rows ? c.skip : VEC, hat, g);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                s[j] = __fmaf_rn(g[j], hat[j], s[j]);
                s[VEC + j] += g[j];
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 2 * VEC; ++j) {
        s[j] = over_slab(s[j]);
        if (threadIdx.x % 64 < kSlab) sums[threadIdx.x / 64][lane][j] = s[j];
    }
    __syncthreads();
    const int i = int(threadIdx.x), which = i / (kSlab * VEC), at = i % (kSlab * VEC), j = at % VEC;
    void *out = which ? b.dbias : b.dweight;
    if (which > 1 || !out) return;
    const Columns<VEC> o(int64_t(blockIdx.x) * kSlab + at / VEC, a.width);
    if (j < o.skip) return;
    float v = sums[0][at / VEC][which * VEC + j];
#pragma unroll
    for (int w = 1; w < kSmallThreads / 64; ++w) v += sums[w][at / VEC][which * VEC + j];
    put_gradient(a, b, out, o.col + j, v);
}

// dx of rows in the registers of T threads, four vectors each.
template <int X, int Y, int T, int VEC>
__device__ __forceinline__ void small_rows(const LayerArgs &a, const LayerBackward &b, int block)
{
    constexpr int U = 4;
    const int t = int(threadIdx.x) % T;
    const int64_t row = int64_t(block) * (kSmallThreads / T) + group_of<T>();
    if (row >= a.rows) return;   // no thread of another row waits for these
    Rows<X, Y, T, U, 1, VEC> in;
    in.template load_as<false>(a, b, row, t);
    auto &[z, dz, dy, mean, rstd] = in;
    float s[2] = {0.0f, 0.0f};
    float hat[U][VEC], d[U][VEC];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Columns<VEC> c(u * T + t, a.width);
        float w[VEC];
        load_weight<VEC>(b.weight, a.weight_dtype, c.col, 1.0f, w);
        normalise<X, Y, VEC>(z[0][u], dy[0][u], mean[0], rstd[0], c.skip, hat[u], d[u]);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            d[u][j] *= w[j];
            s[0] += d[u][j];
            s[1] = __fmaf_rn(d[u][j], hat[u][j], s[1]);
        }
    }
    int turn = 0;
    row_sum<T, kSmallThreads>(s, turn);
    const Along k(s[0], s[1], a);
    void *dx = row_of<X>(b.dx, row, a.x_stride);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Columns<VEC> c(u * T + t, a.width);
        float v[VEC];
        dx_of<X, VEC>(k, rstd[0], d[u], hat[u], dz[0][u], v);
        if (c.skip < VEC) store<X, VEC>(dx, c.col, v, c.skip);
    }
}

template <int X, int Y, int T, int VEC>
__global__ void __launch_bounds__(kSmallThreads) layernorm_grad_small(LayerArgs a, LayerBackward b, int slabs)
{
    if (int(blockIdx.x) < slabs)
        small_columns<X, Y, VEC>(a, b);
    else
        small_rows<X, Y, T, VEC>(a, b, int(blockIdx.x) - slabs);
}

template <int X, int Y, int T, int VEC>
hipError_t run_small(const LayerArgs &a, const LayerBackward &b, hipStream_t s)
{
    const int64_t each = kSmallThreads / T, slabs = (a.width + kSlab * VEC - 1) / (kSlab * VEC);
    const dim3 g(static_cast<unsigned>(slabs + (b.dx ? (a.rows + each - 1) / each : 0)));
    hipLaunchKernelGGL((layernorm_grad_small<X, Y, T, VEC>), g, dim3(kSmallThreads), 0, s, a, b, int(slabs));
    return hipGetLastError();
}

template <int X, int Y, int THREADS, int T, int U, int R, bool AHEAD, int VEC>
hipError_t run_grad(const LayerArgs &a, const LayerBackward &b, hipStream_t s)
{
    constexpr int vectors = U == 1 ? T : T * U - T / 2 + 1;   // of a row that it is for
    constexpr RowPlan plan = row_plan(vectors, VEC, THREADS < 512);
    static_assert(plan.threads == THREADS && plan.rows == THREADS / T * R,
                  "the parts are planned for it");
    hipLaunchKernelGGL((layernorm_grad_rows<X, Y, THREADS, T, U, R, AHEAD, VEC>), dim3(b.n_parts), dim3(THREADS), 0, s,
                       a, b);
    return hipGetLastError();
}

// Rows of up to 256 vectors, a vector a thread. Half as many workgroups of twice
// the threads leave half the parts: 2048 rows of 1024 fp32 values 9.5 us against
// 11.2, 2^21 bf16 values in rows of 1024 8.7 against 10.4. Where the rows come from
// memory, smaller workgroups that do not wait for each other do better: 32768 rows
// of 2048 bf16 values 92 us against 97, 768 columns 106 against 119.
template <int X, int Y, int T, int VEC>
hipError_t run_narrow(const LayerArgs &a, const LayerBackward &b, hipStream_t s)
{
    return a.stream ? run_grad<X, Y, 256, T, 1, 2, true, VEC>(a, b, s) : run_grad<X, Y, 512, T, 1, 2, true, VEC>(a, b, s);
}

}  // namespace

hipError_t launch_layernorm_rows(const LayerArgs &a, const LayerBackward &b, hipStream_t s)
{
    return by_types(a, [&](auto x, auto y) {
        constexpr int X = x(), Y = y(), VEC = layer_vector(X, Y);
        if (a.width < VEC) return run_narrow<X, Y, 8, 1>(a, b, s);
        const int64_t vectors = (a.width + VEC - 1) / VEC;
        if (vectors <= 8) return run_narrow<X, Y, 8, VEC>(a, b, s);
        if (vectors <= 16) return run_narrow<X, Y, 16, VEC>(a, b, s);
        if (vectors <= 32) return run_narrow<X, Y, 32, VEC>(a, b, s);
        if (vectors <= 64) return run_narrow<X, Y, 64, VEC>(a, b, s);
        // three vectors a thread where one would leave threads idle, and then no
        // barrier: 2^26 bf16 values in rows of 768 95 us against 105, of 1536 98
        // against 106; 2^21 in rows of 1536 11.5 against 11.9. One vector a thread by
        // three waves 107 and 14.8; fp32 rows of 384 and 768 183 to 186 us either way
        if (vectors <= 96 && a.stream) return run_grad<X, Y, 256, 32, 3, 1, true, VEC>(a, b, s);
        if (vectors <= 128) return run_narrow<X, Y, 128, VEC>(a, b, s);
        if (vectors <= 192)
            return a.stream ? run_grad<X, Y, 256, 64, 3, 1, true, VEC>(a, b, s)
                            : run_grad<X, Y, 512, 64, 3, 1, true, VEC>(a, b, s);
        if (vectors <= 256) return run_narrow<X, Y, 256, VEC>(a, b, s);
        // rows read past the caches by workgroups of three waves: 2^26 bf16 values in
        // rows of 2560 102 us against 122, of 2880 101 against 115; fp32 rows of 1280
        // 179 to 185 against 190, but of 1440 199 against 181
        if (vectors <= (VEC == 4 ? 320 : 384) && a.stream) return run_grad<X, Y, 192, 192, 2, 1, true, VEC>(a, b, s);
        // two vectors a thread of 256 against one of 512: 8191 rows of 2047 fp32
        // values 37 us against 47, 2^26 bf16 values in rows of 4096 95 against 102,
        // 2^21 13.7 against 11.3
        if (vectors <= 512) return run_grad<X, Y, 512, 256, 2, 1, true, VEC>(a, b, s);
        if (vectors <= 1024) return run_grad<X, Y, 512, 512, 2, 1, true, VEC>(a, b, s);
        // 2^26 bf16 values in rows of 12288 105 us, with four vectors a thread 138 and
        // without the next row ahead 114; fp32 rows of 5120 178, 205 and 198
        if (vectors <= 1536) return run_grad<X, Y, 512, 512, 3, 1, true, VEC>(a, b, s);
        // 2^26 bf16 values in rows of 16384 131 us, with all 256 registers taken and
        // 16 to 19 spilled; by 1024 threads with two vectors each, which leaves them
        // half the registers, 165
        return run_grad<X, Y, 512, 512, 4, 1, false, VEC>(a, b, s);
    });
}

hipError_t launch_layernorm_small(const LayerArgs &a, const LayerBackward &b, hipStream_t s)
{
    return by_types(a, [&](auto x, auto y) {
        constexpr int X = x(), Y = y(), VEC = layer_vector(X, Y);
        if (a.width < VEC) return run_small<X, Y, 64, 1>(a, b, s);
        // a wave a row, or a workgroup
        return a.width <= 256 * VEC ? run_small<X, Y, 64, VEC>(a, b, s) : run_small<X, Y, 512, VEC>(a, b, s);
    });
}

hipError_t launch_layernorm_wide(const LayerArgs &a, const LayerBackward &b, hipStream_t s)
{
    return by_types(a, [&](auto x, auto y) {
        constexpr int X = x(), Y = y(), VEC = layer_vector(X, Y);
        hipError_t e = hipSuccess;
        // the sums first: dx may take dy's place
        if (b.parts) {
            const dim3 g(static_cast<unsigned>((a.width + 64 * VEC - 1) / (64 * VEC)), static_cast<unsigned>(b.n_parts));
            hipLaunchKernelGGL((layernorm_grad_columns<X, Y, VEC>), g, dim3(256), 0, s, a, b);
            e = hipGetLastError();
        }
        for (int64_t first = 0; b.dx && e == hipSuccess && first < a.rows; first += kMostGroups) {
            const dim3 g(static_cast<unsigned>(std::min(kMostGroups, a.rows - first)));
            hipLaunchKernelGGL((layernorm_grad_wide<X, Y, VEC>), g, dim3(1024), 0, s, a, b, first);
            e = hipGetLastError();
        }
        return e;
    });
}

hipError_t launch_layernorm_join(const LayerArgs &a, const LayerBackward &b, hipStream_t s)
{
    const dim3 g(static_cast<unsigned>((a.width + kJoinColumns - 1) / kJoinColumns), b.dbias ? 2 : 1);
    hipLaunchKernelGGL(layernorm_grad_join, g, dim3(kJoinColumns * kJoinSlices), 0, s, a, b);
    return hipGetLastError();
}

}  // namespace ddp
