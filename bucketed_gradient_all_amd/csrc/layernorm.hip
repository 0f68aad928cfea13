// The layer norm's forward pass.
//
//   z    = R(x + add), or x
//   mean = sum z / H                          0 for DDP_RMS_NORM
//   rstd = 1 / sqrt(sum (z - mean)^2 / H + eps)
//   y    = R((z - mean) * rstd * weight + bias)
//
// One pass over memory: a row stays in the registers of a few lanes, a wave or a
// workgroup between its statistics and its output, so the kernel is bound by
// memory: 32768 rows of 2048 bf16 values with residual 87 us (6.2 TB/s), 16384
// rows of 1024 fp32 values 46 us (5.8 TB/s), 8 rows 3 us in a graph, a launch's
// own time. Sums are fp32 over the row's threads, then over the wave by cross-lane
// adds.
//   * The mean is corrected: sum (z - m) / H for the rounded mean m of the first
//     sum is added to it, and taken off the squares' sum. It costs one addition
//     an element and keeps rows exact that lie far from zero.
#include "layernorm_kernels.h"

namespace ddp {
namespace {

// z's columns from x's and add's.
template <int X, int VEC, bool STREAM = false>
__device__ __forceinline__ void load_z(const LayerForward &f, const void *x, const void *add, const Columns<VEC> &c,
                                       float (&v)[VEC])
{
    widen_all<X, VEC>(load<X, VEC, STREAM>(x, c.col), v);
    if (f.add) {
        float w[VEC];
        widen_all<X, VEC>(load<X, VEC, STREAM>(add, c.col), w);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] = widen<X>(narrow<X>(v[j] + w[j]));
    }
}

// The mean's correction and the deviation from a row's second sums.
struct Stats {
    float shift;   // added to the rounded mean
    float rstd;
    __device__ __forceinline__ Stats(float sum, float squares, const LayerArgs &a)
    {
        const float h = float(a.width);
        shift = a.rms ? 0.0f : sum / h;
        const float variance = squares / h - shift * shift;
        rstd = 1.0f / sqrtf((variance < 0.0f ? 0.0f : variance) + a.eps);   // a NaN stays one
    }
};

// Threads of a workgroup whose rows are shared by T threads each: 256, or T.
constexpr int threads_of(int t)
{
    return t <= 64 ? 256 : t;
}

// A row in the registers of T threads, U vectors each.
template <int X, int Y, int T, int U, int VEC>
__global__ void __launch_bounds__(threads_of(T)) layernorm_rows(LayerArgs a, LayerForward f, int64_t first)
{
    constexpr int THREADS = threads_of(T);
    const int64_t row = first + int64_t(blockIdx.x) * (THREADS / T) + group_of<T>();
    if (row >= a.rows) return;   // no thread of another row waits for these
    const int t = int(threadIdx.x) % T;
    const void *x = row_of<X>(f.x, row, a.x_stride), *add = row_of<X>(f.add, row, a.add_stride);
    float v[U][VEC];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Columns<VEC> c(u * T + t, a.width);
        if (a.stream)
            load_z<X, VEC, true>(f, x, add, c, v[u]);
        else
            load_z<X, VEC>(f, x, add, c, v[u]);
    }
    if (f.z) {
        void *z = row_of<X>(f.z, row, a.z_stride);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const Columns<VEC> c(u * T + t, a.width);
            if (c.skip < VEC) store<X, VEC>(z, c.col, v[u], c.skip);
        }
    }
    int turn = 0;
    float mean = 0.0f;
    if (!a.rms) {
        float s[1] = {0.0f};
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const Columns<VEC> c(u * T + t, a.width);
#pragma unroll
            for (int j = 0; j < VEC; ++j) s[0] += j >= c.skip ? v[u][j] : 0.0f;
        }
        row_sum<T, THREADS>(s, turn);
        mean = s[0] / float(a.width);
    }
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Columns<VEC> c(u * T + t, a.width);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            v[u][j] = j >= c.skip ? v[u][j] - mean : 0.0f;
            s[0] += v[u][j];
            s[1] = __fmaf_rn(v[u][j], v[u][j], s[1]);
        }
    }
    row_sum<T, THREADS>(s, turn);
    const Stats k(s[0], s[1], a);
    if (t == 0) {
        if (f.mean) ((GLOBAL float *)f.mean)[row] = mean + k.shift;
        if (f.rstd) ((GLOBAL float *)f.rstd)[row] = k.rstd;
    }
    void *y = row_of<Y>(f.y, row, a.y_stride);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Columns<VEC> c(u * T + t, a.width);
        float w[VEC], b[VEC];
        load_weight<VEC>(f.weight, a.weight_dtype, c.col, 1.0f, w);
        load_weight<VEC>(f.bias, a.weight_dtype, c.col, 0.0f, b);
#pragma unroll
        for (int j = 0; j < VEC; ++j) w[j] = __fmaf_rn((v[u][j] - k.shift) * k.rstd, w[j], b[j]);
        if (c.skip < VEC) store<Y, VEC>(y, c.col, w, c.skip);
    }
}

// A row of any width by a workgroup, read again for each pass: from z once it
// is written, which may lie where x or add does. A thread uses only columns
// that it wrote itself. Its sums are 64 bits: they may be long.
template <int X, int Y, int VEC>
__global__ void __launch_bounds__(1024) layernorm_wide(LayerArgs a, LayerForward f, int64_t first)
{
    constexpr int T = 1024, THREADS = T;
    const int64_t row = first + blockIdx.x;
    const void *x = row_of<X>(f.x, row, a.x_stride), *add = row_of<X>(f.add, row, a.add_stride);
    void *z = f.z ? row_of<X>(f.z, row, a.z_stride) : nullptr;
    const int64_t vectors = (a.width + VEC - 1) / VEC;
    const auto again = [&](const Columns<VEC> &c, float (&v)[VEC]) {
        if (z)
            widen_all<X, VEC>(load<X, VEC>(z, c.col), v);
        else
            load_z<X, VEC>(f, x, add, c, v);
    };
    int turn = 0;
    float v[VEC];
    float m[1] = {0.0f};
    if (z || !a.rms) {
        double sum = 0.0;
        for (int64_t i = threadIdx.x; i < vectors; i += T) {
            const Columns<VEC> c(i, a.width);
            load_z<X, VEC>(f, x, add, c, v);
            if (z) store<X, VEC>(z, c.col, v, c.skip);
#pragma unroll
            for (int j = 0; j < VEC; ++j) sum += j >= c.skip ? double(v[j]) : 0.0;
        }
        m[0] = float(sum);
        row_sum<T, THREADS>(m, turn);
    }
    const float mean = a.rms ? 0.0f : m[0] / float(a.width);
    double sum = 0.0, squares = 0.0;
    for (int64_t i = threadIdx.x; i < vectors; i += T) {
        const Columns<VEC> c(i, a.width);
        again(c, v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const double d = j >= c.skip ? double(v[j] - mean) : 0.0;
            sum += d;
            squares = __fma_rn(d, d, squares);
        }
    }
    float s[2] = {float(sum), float(squares)};
    row_sum<T, THREADS>(s, turn);
    const Stats k(s[0], s[1], a);
    if (threadIdx.x == 0) {
        if (f.mean) ((GLOBAL float *)f.mean)[row] = mean + k.shift;
        if (f.rstd) ((GLOBAL float *)f.rstd)[row] = k.rstd;
    }
    void *y = row_of<Y>(f.y, row, a.y_stride);
    for (int64_t i = threadIdx.x; i < vectors; i += T) {
        const Columns<VEC> c(i, a.width);
        float w[VEC], b[VEC];
        again(c, v);
        load_weight<VEC>(f.weight, a.weight_dtype, c.col, 1.0f, w);
        load_weight<VEC>(f.bias, a.weight_dtype, c.col, 0.0f, b);
#pragma unroll
        for (int j = 0; j < VEC; ++j) w[j] = __fmaf_rn((v[j] - mean - k.shift) * k.rstd, w[j], b[j]);
        store<Y, VEC>(y, c.col, w, c.skip);
    }
}

// A launch covers rows in order, as many as its grid holds.
template <class F>
hipError_t over_rows(int64_t rows, int64_t each, F &&launch)
{
    for (int64_t first = 0; first < rows; first += kMostGroups * each) {
        launch(dim3(static_cast<unsigned>(std::min(kMostGroups, (rows - first + each - 1) / each))), first);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <int X, int Y, int T, int U, int VEC>
hipError_t run_rows(const LayerArgs &a, const LayerForward &f, hipStream_t s)
{
    return over_rows(a.rows, threads_of(T) / T, [&](dim3 g, int64_t first) {
        hipLaunchKernelGGL((layernorm_rows<X, Y, T, U, VEC>), g, dim3(threads_of(T)), 0, s, a, f, first);
    });
}

}  // namespace

// Whether rows of 2049 to 8192 vectors are read again for each pass instead of kept
// in registers, four or eight vectors a thread. Where a row has few more vectors
// than the next smaller count holds, half of the threads' registers stay empty, and
// reading x again from L2 costs less; not with 256 rows or fewer, where each CU has
// one and waits for it three times. Of 2^26 elements without add, kept and read
// again: 16-bit rows of 16392 columns 112 and 88 us, of 28000 88 and 86, of 30000 83
// and 86 (320 rows: 13.3 and 10.8, 14.0 and 14.8, 14.4 and 15.4; 256 rows 8.1 and
// 8.3, 8.3 and 10.6); fp32 rows of 8200 158 and 135, of 11000 135 and 135, of 12000
// 128 and 134; into 16 bits of 16400 133 and 126, of 20000 124 and 125, but into fp32
// of 18000 93 and 99 (2560 rows). With add all passes but the first read z: 16-bit
// rows past the caches of 16392 165 and 148, of 20000 149 and 141, of 22000 141 and
// 143; from the caches 37 and 38, fp32 ones of 8200 230 and 257.
bool reads_again(const LayerArgs &a, const LayerForward &f, int64_t vectors, int vec)
{
    if (f.add) return vec == 8 && a.stream && f.z && vectors <= 2600;
    if (a.rows <= 256) return false;
    if (vec == 8) return vectors <= 3500;
    return vectors <= 2700 || (a.y_dtype != DDP_F32 && vectors > 4096 && vectors <= 4500);
}

// A vector a thread, or two where that makes more waves than it saves: of 2^26
// elements with weight and bias, 1024 16-bit columns take 92 us by one wave with
// two vectors and 95 by two with one, 512 fp32 columns 186 and 173; 4096 16-bit
// columns 143 us by one wave with eight, 101 by four with two, 100 by eight with
// one; 8192 109 by four with four, 101 by eight with two, 110 by sixteen with one.
// Up to 32768 columns in registers: with add 16384 fp32 ones 206 us, 252 read
// again; 32768 16-bit ones 122 and 141.
// Where those counts leave a fifth of the threads idle or more, a count nearer to the
// row: 768 16-bit columns 95 us by half a wave with three vectors (where they come
// from memory; 5.7 us against 5.3 for 2^21 elements) and 100 by a wave with two, 1536
// 101 by three waves and 106 by four, 2560 109 by five and 126 by eight; 1280 fp32
// columns 181 and 198; 5120 16-bit ones 105 and 119, 10240 116 and 122, 12288 108 and
// 113. Twelve waves for 6144 gained nothing.
// Narrow rows share a wave: 256 16-bit columns 91 us, 145 with a wave each.
hipError_t launch_layernorm(const LayerArgs &a, const LayerForward &f, hipStream_t s)
{
    return by_types(a, [&](auto x, auto y) {
        constexpr int X = x(), Y = y(), VEC = layer_vector(X, Y);
        if (a.width < VEC) return run_rows<X, Y, 8, 1, 1>(a, f, s);
        const int64_t vectors = (a.width + VEC - 1) / VEC;
        if (vectors <= 8) return run_rows<X, Y, 8, 1, VEC>(a, f, s);
        if (vectors <= 16) return run_rows<X, Y, 16, 1, VEC>(a, f, s);
        if (vectors <= 32) return run_rows<X, Y, 32, 1, VEC>(a, f, s);
        if (vectors <= 64) return run_rows<X, Y, 64, 1, VEC>(a, f, s);
        if constexpr (VEC == 8) {
            if (vectors <= 96 && a.stream) return run_rows<X, Y, 32, 3, VEC>(a, f, s);
        }
        if (vectors <= 128) return run_rows<X, Y, VEC == 4 ? 128 : 64, VEC == 4 ? 1 : 2, VEC>(a, f, s);
        if (vectors <= 192) return run_rows<X, Y, 192, 1, VEC>(a, f, s);
        if (vectors <= 256) return run_rows<X, Y, 256, 1, VEC>(a, f, s);
        if (vectors <= 320) return run_rows<X, Y, 320, 1, VEC>(a, f, s);
        if (vectors <= 512) return run_rows<X, Y, 512, 1, VEC>(a, f, s);
        if (vectors <= 640) return run_rows<X, Y, 320, 2, VEC>(a, f, s);
        if (vectors <= 1024) return run_rows<X, Y, 512, 2, VEC>(a, f, s);
        if (vectors <= 1280) return run_rows<X, Y, 640, 2, VEC>(a, f, s);
        if (vectors <= 1536) return run_rows<X, Y, 768, 2, VEC>(a, f, s);
        if (vectors <= 2048) return run_rows<X, Y, 1024, 2, VEC>(a, f, s);
        if (!reads_again(a, f, vectors, VEC)) {
            if (vectors <= 4096) return run_rows<X, Y, 1024, 4, VEC>(a, f, s);
            if (VEC == 4 && vectors <= 8192) return run_rows<X, Y, 1024, VEC == 4 ? 8 : 4, VEC>(a, f, s);
        }
        return over_rows(a.rows, 1, [&](dim3 g, int64_t first) {
            hipLaunchKernelGGL((layernorm_wide<X, Y, VEC>), g, dim3(1024), 0, s, a, f, first);
        });
    });
}

}  // namespace ddp
