// Orthogonalised updates of matrices with a side of up to 64, whole stacks at a
// time.  All steps' factors are polynomials of S = G G^T / (|G| + eps)^2, m x m
// for the smaller side m, so the steps need not touch the rows: with P_t = a I +
// b S_t + c S_t^2 and S_{t+1} = P_t S_t P_t,
//   O = (P_last ... P_0) G / (|G| + eps),    |G|^2 = the trace of G G^T.
// Three launches, G read twice: 16 matrices of 16 x 4096 float take 5, 9 and 5 us,
// bound by the launches and by small_steps' chain of products in one workgroup (4.2
// MB of G: 0.9 us; sixteen launches of steps on tiles would take 80).  16 of 32 x 4096
// take 9, 21 and 11 us, of 64 x 4096 24, 90 and 35: there the chain is most of it.  S loses what
// is below its own rounding, and each step multiplies that by up to a^2, so this is
// done in double throughout: the double matrix instruction (16 x 16, sums of 4),
// whose work is small here (16 x 4096: 2 MFLOP a matrix).  Its operands: lane l holds
// element l / 16 of row l % 16; results: rows l / 16 + 4 r of column l % 16, r = 0 .. 3.
#include <algorithm>
#include <cmath>

#include "kernels.h"
#include "orthogonalize.h"

namespace sgemm {
namespace {

typedef double v4d __attribute__((ext_vector_type(4)));

template <int TYPE>
__device__ __forceinline__ double load_as(const void* p, int64_t i) {
    if constexpr (TYPE == T_F32) return static_cast<const float*>(p)[i];
    else if constexpr (TYPE == T_F16) return float(static_cast<const _Float16*>(p)[i]);
    else return float(static_cast<const __bf16*>(p)[i]);
}
template <int TYPE>
__device__ __forceinline__ void store_as(void* p, int64_t i, double v) {
    if constexpr (TYPE == T_F32) static_cast<float*>(p)[i] = float(v);
    else if constexpr (TYPE == T_F16) static_cast<_Float16*>(p)[i] = _Float16(float(v));
    else static_cast<__bf16*>(p)[i] = __bf16(float(v));
}

// (A template, as the host pass does not know the builtin.)
template <int>
__device__ __forceinline__ v4d mma(double a, double b, v4d c) {
    return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0);
}

// Partial sums of G G^T (of G^T G for a tall G), blocks of 16 x 16 of a side of 16
// MB: share x of matrix y, its four waves' sums added in order.
template <int TYPE, int MB>
__global__ void __launch_bounds__(256) small_gram(const void* G, bool tall, int m, int64_t n, int64_t ldg, int64_t sg,
                                                  int64_t share, double* out) {
    constexpr int SIDE = 16 * MB;
    __shared__ double sum[SIDE * SIDE];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
    const int64_t b = blockIdx.y, c0 = blockIdx.x * share, c1 = c0 + share < n ? c0 + share : n;
    v4d acc[MB][MB];
#pragma unroll
    for (int x = 0; x < MB; x++)
#pragma unroll
        for (int y = 0; y < MB; y++) acc[x][y] = v4d{0, 0, 0, 0};
    // Four columns a lane group at a time, four groups, four waves.
    for (int64_t c = c0 + 16 * wave; c < c1; c += 64) {
        double v[MB][4];
#pragma unroll
        for (int x = 0; x < MB; x++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int64_t r = 16 * x + i, col = tall ? c + 4 * e + g : c + 4 * g + e;
                const bool in = r < m && col < c1;
                const int64_t at = in ? (tall ? col * ldg + r : r * ldg + col) : 0;
                v[x][e] = load_as<TYPE>(G, b * sg + at);
                if (!in) v[x][e] = 0.0;
            }
#pragma unroll
        for (int e = 0; e < 4; e++)
#pragma unroll
            for (int x = 0; x < MB; x++)
#pragma unroll
                for (int y = 0; y < MB; y++) acc[x][y] = mma<0>(v[x][e], v[y][e], acc[x][y]);
    }
    for (int w = 0; w < 4; w++) {
        if (wave == w) {
#pragma unroll
            for (int x = 0; x < MB; x++)
#pragma unroll
                for (int y = 0; y < MB; y++)
#pragma unroll
                    for (int r = 0; r < 4; r++) {
                        double* const at = &sum[(16 * x + 4 * r + g) * SIDE + 16 * y + i];
                        *at = w ? *at + acc[x][y][r] : acc[x][y][r];
                    }
        }
        __syncthreads();
    }
    double* const to = out + (b * gridDim.x + blockIdx.x) * SIDE * SIDE;
    for (int e = threadIdx.x; e < SIDE * SIDE; e += 256) to[e] = sum[e];
}

// From the partial sums the product of all steps' factors over |G| + eps, a
// matrix a workgroup.  Every matrix here is a polynomial of one symmetric matrix: a
// row serves as a column, and products commute.
template <int MB>
__global__ void __launch_bounds__(256) small_steps(const double* parts, int shares, int m, double eps, int steps,
                                                   const SmallCoefficients coef, double* out) {
    constexpr int SIDE = 16 * MB, LD = SIDE + 2;
    __shared__ double S[SIDE * LD], P[SIDE * LD], Q[SIDE * LD], T[SIDE * LD];
    __shared__ double trace;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
    const double* const from = parts + int64_t(blockIdx.x) * shares * SIDE * SIDE;
    for (int e = threadIdx.x; e < SIDE * SIDE; e += 256) {
        double v = 0;
#pragma unroll 4
        for (int s = 0; s < shares; s++) v += from[s * SIDE * SIDE + e];
        S[e / SIDE * LD + e % SIDE] = v;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        double v = 0;
        for (int r = 0; r < m; r++) v += S[r * LD + r];
        trace = v;
    }
    __syncthreads();
    // 0 for zeros, whatever eps (f^2 may pass the largest double), NaN stays.
    const double f = trace > 0 ? 1.0 / (sqrt(trace) + eps) : trace;
    for (int e = threadIdx.x; e < SIDE * SIDE; e += 256) S[e / SIDE * LD + e % SIDE] *= f * f;
    // C = A B, waves by blocks; `put` takes each element.
    auto product = [&](const double* A, const double* B, auto put) {
        __syncthreads();
        for (int t = wave; t < MB * MB; t += 4) {
            const int x = t / MB, y = t % MB;
            v4d acc = {0, 0, 0, 0};
#pragma unroll 4
            for (int k = 0; k < SIDE / 4; k++)
                acc = mma<0>(A[(16 * x + i) * LD + 4 * k + g], B[(16 * y + i) * LD + 4 * k + g], acc);
#pragma unroll
            for (int r = 0; r < 4; r++) put(16 * x + 4 * r + g, 16 * y + i, acc[r]);
        }
        __syncthreads();
    };
#pragma unroll 1
    for (int t = 0; t < steps; t++) {
        const double a = coef.v[3 * t], b = coef.v[3 * t + 1], c = coef.v[3 * t + 2];
        product(S, S, [&](int r, int q, double v) {
            P[r * LD + q] = c * v + b * S[r * LD + q] + (r == q && r < m ? a : 0.0);
        });
        if (t == 0) {
            for (int e = threadIdx.x; e < SIDE * LD; e += 256) Q[e] = P[e];
        } else {
            product(P, Q, [&](int r, int q, double v) { T[r * LD + q] = v; });
            for (int e = threadIdx.x; e < SIDE * LD; e += 256) Q[e] = T[e];
        }
        if (t + 1 == steps) break;
        product(P, S, [&](int r, int q, double v) { T[r * LD + q] = v; });
        product(T, P, [&](int r, int q, double v) { S[r * LD + q] = v; });
    }
    __syncthreads();
    double* const to = out + int64_t(blockIdx.x) * SIDE * SIDE;
    for (int e = threadIdx.x; e < SIDE * SIDE; e += 256) to[e] = Q[e / SIDE * LD + e % SIDE] * f;
}

// O = Q G (G Q for a tall G): 64 columns (rows) of matrix y a workgroup, 16 a wave.
template <int TYPE, int MB>
__global__ void __launch_bounds__(256) small_apply(const double* Qs, const void* G, bool tall, int m, int64_t n,
                                                   int64_t ldg, int64_t sg, void* O, int64_t ldo, int64_t so) {
    constexpr int SIDE = 16 * MB;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
    const double* const Q = Qs + int64_t(blockIdx.y) * SIDE * SIDE;
    const int64_t b = blockIdx.y, c0 = (int64_t(blockIdx.x) * 4 + wave) * 16, c = c0 + i;
    if (c0 >= n) return;
    double v[SIDE / 4];  // G's element k = 4 u + g of column c
#pragma unroll
    for (int u = 0; u < SIDE / 4; u++) {
        const int64_t k = 4 * u + g;
        const bool in = k < m && c < n;
        v[u] = load_as<TYPE>(G, b * sg + (in ? (tall ? c * ldg + k : k * ldg + c) : 0));
        if (!in) v[u] = 0.0;
    }
#pragma unroll
    for (int x = 0; x < MB; x++) {
        v4d acc = {0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < SIDE / 4; u++) {
            const double q = Q[(16 * x + i) * SIDE + 4 * u + g];
            acc = tall ? mma<0>(v[u], q, acc) : mma<0>(q, v[u], acc);
        }
#pragma unroll
        for (int r = 0; r < 4; r++) {
            // Wide: row 16 x + 4 r + g of column c; tall: column 16 x + i of row c0 + 4 r + g.
            const int64_t row = tall ? c0 + 4 * r + g : 16 * x + 4 * r + g, col = tall ? 16 * x + i : c;
            if (row < (tall ? n : m) && col < (tall ? m : n)) store_as<TYPE>(O, b * so + row * ldo + col, acc[r]);
        }
    }
}

// Columns of a workgroup's share of the sums, and the shares.
int64_t small_share(int64_t n) { return std::max<int64_t>(256, ceil_div(ceil_div(n, 16), 64) * 64); }

template <int TYPE, int MB>
hipError_t run(const OrthoArgs& g, hipStream_t s) {
    constexpr int SIDE = 16 * MB;
    const bool tall = g.M > g.N;
    const int m = int(std::min(g.M, g.N));
    const int64_t n = std::max(g.M, g.N), share = small_share(n);
    const int shares = int(ceil_div(n, share));
    const unsigned batch = unsigned(g.batch);
    double* const Q = static_cast<double*>(g.ws);
    double* const parts = Q + g.batch * SIDE * SIDE;
    SmallCoefficients coef;
    for (int i = 0; i < 3 * g.steps; i++) coef.v[i] = g.coef[i];
    hipLaunchKernelGGL((small_gram<TYPE, MB>), dim3(shares, batch), dim3(256), 0, s, g.G, tall, m, n, g.ldg, g.sg, share, parts);
    hipLaunchKernelGGL((small_steps<MB>), dim3(batch), dim3(256), 0, s, parts, shares, m, g.eps, g.steps, coef, Q);
    hipLaunchKernelGGL((small_apply<TYPE, MB>), dim3(unsigned(ceil_div(n, 64)), batch), dim3(256), 0, s, Q, g.G, tall, m, n,
                       g.ldg, g.sg, g.O, g.ldo, g.so);
    return hipGetLastError();
}

template <int TYPE>
hipError_t by_side(const OrthoArgs& g, hipStream_t s) {
    const int64_t m = std::min(g.M, g.N);
    if (m <= 16) return run<TYPE, 1>(g, s);
    if (m <= 32) return run<TYPE, 2>(g, s);
    return run<TYPE, 4>(g, s);
}

}  // namespace

size_t ortho_small_bytes(int64_t batch, int64_t M, int64_t N) {
    const int64_t m = std::min(M, N), side = m <= 16 ? 16 : m <= 32 ? 32 : 64, n = std::max(M, N);
    return size_t(batch) * side * side * sizeof(double) * size_t(1 + ceil_div(n, small_share(n)));
}

hipError_t launch_ortho_small(const OrthoArgs& g, hipStream_t s) {
    if (g.type == T_F32) return by_side<T_F32>(g, s);
    if (g.type == T_F16) return by_side<T_F16>(g, s);
    return by_side<T_BF16>(g, s);
}

}  // namespace sgemm
