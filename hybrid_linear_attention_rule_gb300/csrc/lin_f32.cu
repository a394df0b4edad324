// lin_f32.cu -- linear attention's jobs (lin.cuh) on the CUDA cores, everything in FP32: the path of FP32 inputs.
//
// A CTA holds a [a, 32] slice of one head's state in shared memory and walks the sequence, or a piece of it, in chunks of 32 tokens, a token a
// lane for the decays; the next chunk's rows are on their way, in registers, meanwhile.  The four products of a chunk (x y^T, its
// product with z, x S, y^T z) are register tiles of 4 to 16 accumulators fed by 16-byte shared loads; the scores are worked out again by
// each slice of b.  What bounds it is the shared loads, some 5 for 16 products of a thread, and the sequence of its steps.
#include "lin.cuh"

namespace k3kda {
namespace lin {
namespace {

constexpr int C = 32, THREADS = 256, PITCH_S = kSlice + 4, LEAST = 2;

struct Layout {
    int pa, x, y, z, s, p, w, total;       // floats
    __host__ __device__ explicit Layout(int a) {
        pa = a + 4;
        x = 0;
        y = x + C * pa;
        s = y + C * pa;
        z = s + a * PITCH_S;
        p = z + C * PITCH_S;
        w = p + C * (C + 1);
        total = w + 5 * C;
    }
};

// Pieces of each sequence, where there are fewer CTAs than the GPU holds: their states come from a first pass (STATES), which takes those
// of every piece but the last from zero, and a piece's own chain of those before it.
struct Cut {
    int pieces;
    float *state, *keep;       // [jobs][pieces][N H][slices] of [a, 32] and of one; the last piece's holds the first state where it is written over
    bool kept;
};

template <bool STATES> __global__ void __launch_bounds__(THREADS) scan_kernel(const __grid_constant__ Call A, const Cut cut) {
    extern __shared__ float4 smem4[];
    __shared__ unsigned lost;              // tokens of the chunk whose decay is NaN
    const int parts = STATES ? cut.pieces - 1 : cut.pieces, job = blockIdx.z / parts, piece = blockIdx.z % parts;
    const Job &J = A.job[job];
    const int b0 = blockIdx.y * kSlice, a = J.a, nb = min(kSlice, J.b - b0);
    if (b0 >= J.b) return;
    float *sm = reinterpret_cast<float *>(smem4);
    const Layout L(a);
    float *X = sm + L.x, *Y = sm + L.y, *Z = sm + L.z, *S = sm + L.s, *P = sm + L.p;
    float *hi = sm + L.w, *lo = hi + C, *cin = lo + C, *wt = cin + C, *keep = wt + C;
    const int tid = threadIdx.x, n = blockIdx.x / A.H, h = blockIdx.x % A.H;
    int begin, end;
    seq_bounds(A.cu, n, A.T, begin, end);
    const int len = end - begin, chunks = (len + C - 1) / C;
    const int slot = seq_slot(A.slot, A.num_slots, n);
    const size_t state = ((size_t)(slot < 0 ? 0 : slot) * A.H + h) * a * J.b;
    const int tx = tid % 8, ty = tid / 8;

    const int begins = (int)((long long)chunks * piece / cut.pieces), ends = (int)((long long)chunks * (piece + 1) / cut.pieces);
    // a piece's place among the states
    auto place = [&](int p) { return (((size_t)job * cut.pieces + p) * gridDim.x + blockIdx.x) * gridDim.y + blockIdx.y; };
    long long units = 0;                   // STATES: the piece's decay (warp 0)
    unsigned gone = 0;
    if (piece == 0) {
        const float *kept = !STATES && cut.kept && cut.pieces > 1 ? cut.state + place(cut.pieces - 1) * (128 * kSlice) : nullptr;
        for (int i = tid; i < a * kSlice; i += THREADS) {
            const int c = i / kSlice, b = i % kSlice;
            const float v = kept ? kept[i] : J.first && slot >= 0 && b < nb ? J.first[state + (size_t)c * J.sa + (size_t)(b0 + b) * J.sb] : 0.f;
            S[c * PITCH_S + b] = v;
            if (STATES && cut.kept) cut.state[place(cut.pieces - 1) * (128 * kSlice) + i] = v;
        }
    } else {
        float v[128 * kSlice / THREADS];
#pragma unroll
        for (int k = 0; k < 128 * kSlice / THREADS; ++k) v[k] = 0.f;
        if (!STATES)
            for (int p = 0; p < piece; ++p) {
                const float *from = cut.state + place(p) * (128 * kSlice);
                const float e = cut.keep[place(p)];
#pragma unroll
                for (int k = 0; k < 128 * kSlice / THREADS; ++k)
                    if (tid + k * THREADS < a * kSlice) v[k] = fmaf(e, v[k], from[tid + k * THREADS]);
            }
#pragma unroll
        for (int k = 0; k < 128 * kSlice / THREADS; ++k) {
            const int i = tid + k * THREADS;
            if (i < a * kSlice) S[i / kSlice * PITCH_S + i % kSlice] = v[k];
        }
    }
    const size_t base_x = h / J.x.share, base_y = h / J.y.share, base_z = h / J.z.share;
    const size_t hx = A.H / J.x.share, hy = A.H / J.y.share, hz = A.H / J.z.share;

    // A chunk's rows as 16-byte pieces: piece i of x and y is row i / (a / 4), 4 pieces a thread at most; of z row tid / 8.
    constexpr int MOST = C * 128 / 4 / THREADS;
    const int per_row = a / 4, pieces = C * per_row;
    float4 nx[MOST], ny[MOST], nz;
    float ng = 0.f;
    auto fetch = [&](int it) {
        const int chunk = J.reverse ? chunks - 1 - it : it, t0 = begin + chunk * C, valid = min(C, end - t0);
        const float *const px = static_cast<const float *>(J.x.p), *const py = static_cast<const float *>(J.y.p), *const pz = static_cast<const float *>(J.z.p);
        const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < MOST; ++k) {
            const int i = tid + k * THREADS, t = i / per_row, c = i % per_row * 4;
            const bool in = i < pieces && t < valid;
            if (!STATES) nx[k] = in ? *reinterpret_cast<const float4 *>(px + ((size_t)(t0 + t) * hx + base_x) * a + c) : none;
            ny[k] = in ? *reinterpret_cast<const float4 *>(py + ((size_t)(t0 + t) * hy + base_y) * a + c) : none;
        }
        nz = tid / 8 < valid && tid % 8 * 4 < nb ? *reinterpret_cast<const float4 *>(pz + ((size_t)(t0 + tid / 8) * hz + base_z) * J.b + b0 + tid % 8 * 4) : none;
        if (tid < C) ng = tid < valid ? A.g[A.fixed ? h : (size_t)(t0 + tid) * A.H + h] : 0.f;
    };
    if (begins < ends) fetch(begins);
    for (int it = begins; it < ends; ++it) {
        const int chunk = J.reverse ? chunks - 1 - it : it, t0 = begin + chunk * C, valid = min(C, end - t0);
        __syncthreads();
        if (!STATES && J.anchors && !J.reverse && it > 0 && chunk * C % kAnchor == 0) {
            float *to = J.anchors + ((size_t)(anchor_slot(begin, n) + chunk * C / kAnchor - 1) * A.H + h) * a * J.b;
            for (int i = tid; i < a * kSlice; i += THREADS)
                if (i % kSlice < nb) to[(size_t)(i / kSlice) * J.b + b0 + i % kSlice] = S[i / kSlice * PITCH_S + i % kSlice];
        }
#pragma unroll
        for (int k = 0; k < MOST; ++k) {
            const int i = tid + k * THREADS;
            if (i < pieces) {
                if (!STATES) *reinterpret_cast<float4 *>(X + i / per_row * L.pa + i % per_row * 4) = nx[k];
                *reinterpret_cast<float4 *>(Y + i / per_row * L.pa + i % per_row * 4) = ny[k];
            }
        }
        *reinterpret_cast<float4 *>(Z + tid / 8 * PITCH_S + tid % 8 * 4) = nz;
        if (tid < C) {
            const float g = ng;
            long long v = decay_units(g);
#pragma unroll
            for (int o = 1; o < C; o <<= 1) {
                const long long u = __shfl_up_sync(0xffffffffu, v, o);
                if (tid >= o) v += u;
            }
            const long long all = __shfl_sync(0xffffffffu, v, C - 1);
            // a NaN among the decays is in every sum that takes it in, and in no other
            const unsigned bad = __ballot_sync(0xffffffffu, g != g), upto = 0xffffffffu >> (31 - tid);
            const float nan = __int_as_float(0x7fffffff);
            const float2 f = two_floats(v);
            hi[tid] = f.x;
            lo[tid] = f.y;
            const float up = bad & upto ? nan : exp2_units(v), down = bad & ~upto ? nan : exp2_units(all - v);
            cin[tid] = J.sc * (J.reverse ? down : up);
            wt[tid] = J.sw * (tid < valid ? (J.reverse ? up : down) : 0.f);
            if (tid == 0) lost = bad;
            if (tid == 0) *keep = bad ? nan : exp2_units(all);
            if (STATES) {
                units += all;
                gone |= bad;
            }
        }
        __syncthreads();
        if (it + 1 < ends) fetch(it + 1);

        if constexpr (!STATES) {
        {   // scores: 2 x 2 a thread
            const int i0 = tid / 16, j0 = tid % 16;
            float acc[2][2] = {};
            for (int c = 0; c < a; c += 4) {
                const float4 x0 = *reinterpret_cast<float4 *>(X + i0 * L.pa + c), x1 = *reinterpret_cast<float4 *>(X + (i0 + 16) * L.pa + c);
                const float4 y0 = *reinterpret_cast<float4 *>(Y + j0 * L.pa + c), y1 = *reinterpret_cast<float4 *>(Y + (j0 + 16) * L.pa + c);
                acc[0][0] = fmaf(x0.w, y0.w, fmaf(x0.z, y0.z, fmaf(x0.y, y0.y, fmaf(x0.x, y0.x, acc[0][0]))));
                acc[0][1] = fmaf(x0.w, y1.w, fmaf(x0.z, y1.z, fmaf(x0.y, y1.y, fmaf(x0.x, y1.x, acc[0][1]))));
                acc[1][0] = fmaf(x1.w, y0.w, fmaf(x1.z, y0.z, fmaf(x1.y, y0.y, fmaf(x1.x, y0.x, acc[1][0]))));
                acc[1][1] = fmaf(x1.w, y1.w, fmaf(x1.z, y1.z, fmaf(x1.y, y1.y, fmaf(x1.x, y1.x, acc[1][1]))));
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const int i = i0 + 16 * u, j = j0 + 16 * v;
                    float d = (hi[i] - hi[j]) + (lo[i] - lo[j]);
                    if (lost && ((0xffffffffu >> (31 - i)) ^ (0xffffffffu >> (31 - j))) & lost) d = __int_as_float(0x7fffffff);
                    const bool seen = J.reverse ? j >= i : j <= i;
                    P[i * (C + 1) + j] = seen ? J.sp * exp2f(J.reverse ? -d : d) * acc[u][v] : 0.f;
                }
        }
        __syncthreads();

        {   // outputs: token ty, channels 4 tx .. 4 tx + 3
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int c = 0; c < a; c += 4) {
                const float4 x = *reinterpret_cast<float4 *>(X + ty * L.pa + c);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float4 v = *reinterpret_cast<float4 *>(S + (c + u) * PITCH_S + 4 * tx);
                    const float xc = u == 0 ? x.x : u == 1 ? x.y : u == 2 ? x.z : x.w;
                    o.x = fmaf(xc, v.x, o.x);
                    o.y = fmaf(xc, v.y, o.y);
                    o.z = fmaf(xc, v.z, o.z);
                    o.w = fmaf(xc, v.w, o.w);
                }
            }
            const float ci = cin[ty];
            o = make_float4(o.x * ci, o.y * ci, o.z * ci, o.w * ci);
            // (a z that is not seen is left out, not multiplied by 0: it may be infinite)
            for (int j = 0; j < C; ++j) {
                if (J.reverse ? j <= ty : j >= ty) continue;
                const float p = P[ty * (C + 1) + j];
                const float4 z = *reinterpret_cast<float4 *>(Z + j * PITCH_S + 4 * tx);
                o.x = fmaf(p, z.x, o.x);
                o.y = fmaf(p, z.y, o.y);
                o.z = fmaf(p, z.z, o.z);
                o.w = fmaf(p, z.w, o.w);
            }
            const size_t row = (size_t)(t0 + ty) * A.H + h;
            const float v[4] = {o.x, o.y, o.z, o.w};
            if (J.dots) {
                float dot = 0.f;
                if (ty < valid)
                    for (int u = 0; u < 4; ++u)
                        if (4 * tx + u < nb)
                            dot = fmaf(load_elt(J.r.p, ((size_t)(t0 + ty) * (A.H / J.r.share) + h / J.r.share) * J.b + b0 + 4 * tx + u, 0), v[u], dot);
                dot += __shfl_xor_sync(0xffffffffu, dot, 1);
                dot += __shfl_xor_sync(0xffffffffu, dot, 2);
                dot += __shfl_xor_sync(0xffffffffu, dot, 4);
                if (ty < valid && tx == 0) J.dots[(size_t)blockIdx.y * A.T * A.H + row] = dot;
            }
            if (ty < valid) {
                const float p = P[ty * (C + 1) + ty];
                for (int u = 0; u < 4; ++u)
                    if (4 * tx + u < nb) store_elt(J.out, row * J.b + b0 + 4 * tx + u, fmaf(p, Z[ty * PITCH_S + 4 * tx + u], v[u]), J.out_bf16);
            }
        }
        __syncthreads();
        }

        // the state: rows 4 ty .. 4 ty + 3, channels 4 tx .. 4 tx + 3
        if (4 * ty < a) {
            float acc[4][4];
            const float e = *keep;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float4 v = *reinterpret_cast<float4 *>(S + (4 * ty + u) * PITCH_S + 4 * tx);
                acc[u][0] = e * v.x;
                acc[u][1] = e * v.y;
                acc[u][2] = e * v.z;
                acc[u][3] = e * v.w;
            }
            for (int j = 0; j < valid; ++j) {
                const float4 y = *reinterpret_cast<float4 *>(Y + j * L.pa + 4 * ty), z = *reinterpret_cast<float4 *>(Z + j * PITCH_S + 4 * tx);
                const float w = wt[j], yw[4] = {w * y.x, w * y.y, w * y.z, w * y.w};
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    acc[u][0] = fmaf(yw[u], z.x, acc[u][0]);
                    acc[u][1] = fmaf(yw[u], z.y, acc[u][1]);
                    acc[u][2] = fmaf(yw[u], z.z, acc[u][2]);
                    acc[u][3] = fmaf(yw[u], z.w, acc[u][3]);
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
                *reinterpret_cast<float4 *>(S + (4 * ty + u) * PITCH_S + 4 * tx) = make_float4(acc[u][0], acc[u][1], acc[u][2], acc[u][3]);
        }
        if (!STATES && J.anchors && J.reverse && chunk > 0 && chunk * C % kAnchor == 0) {
            __syncthreads();
            float *to = J.anchors + ((size_t)(anchor_slot(begin, n) + chunk * C / kAnchor - 1) * A.H + h) * a * J.b;
            for (int i = tid; i < a * kSlice; i += THREADS)
                if (i % kSlice < nb) to[(size_t)(i / kSlice) * J.b + b0 + i % kSlice] = S[i / kSlice * PITCH_S + i % kSlice];
        }
    }
    __syncthreads();
    if (STATES) {
        for (int i = tid; i < a * kSlice; i += THREADS) cut.state[place(piece) * (128 * kSlice) + i] = S[i / kSlice * PITCH_S + i % kSlice];
        if (tid == 0) cut.keep[place(piece)] = gone ? __int_as_float(0x7fffffff) : exp2_units(units);
        return;
    }
    if (piece < cut.pieces - 1) return;
    for (int i = tid; i < a * kSlice; i += THREADS) {
        const int c = i / kSlice, b = i % kSlice;
        if (b >= nb) continue;
        const float v = S[c * PITCH_S + b];
        if (J.last && slot >= 0) J.last[state + (size_t)c * J.sa + (size_t)(b0 + b) * J.sb] = v;
        if (J.anchors && J.last_anchor)
            J.anchors[((size_t)(anchor_slot(begin, n) + max(0, len - 1) / kAnchor) * A.H + h) * a * J.b + (size_t)c * J.b + b0 + b] = v;
    }
}

std::atomic<uint64_t> g_attr[2];

constexpr int MOST_CTAS = 320, MOST_CUT = 64;

}  // namespace

size_t f32_workspace() { return (size_t)MOST_CTAS * (128 * kSlice + 1) * sizeof(float); }

cudaError_t launch_scan_f32(const Call &c, cudaStream_t s) {
    if (c.N == 0) return cudaSuccess;
    const int most = (int)(Layout(128).total * sizeof(float));
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = smem_attr_once((const void *)scan_kernel<false>, most, g_attr[0]);
    if (e == cudaSuccess) e = smem_attr_once((const void *)scan_kernel<true>, most, g_attr[1]);
    if (e != cudaSuccess) return e;
    int wide = 0, bytes = 0;
    for (int j = 0; j < c.jobs; ++j) {
        wide = max(wide, slices(c.job[j].b));
        bytes = max(bytes, (int)(Layout(c.job[j].a).total * sizeof(float)));
    }
    // Two CTAs an SM, pieces of LEAST chunks or more on average.  (Heads of 128 channels, uncut and cut: 8 heads of 8,192 tokens 1,938 and 479 us,
    // of 1,024 tokens 247 and 79, of 256 tokens 67 and 34, where pieces of 4 chunks took 50; 32 heads of 2,048 tokens 492 and 495; gradients of 8 heads
    // of 8,192 tokens 2,279 and 1,513.)
    const long long ctas = (long long)c.N * c.H * wide * c.jobs, chunks = c.T / C / c.N;
    long long pieces = min((long long)min(2 * sms, MOST_CTAS) / ctas, chunks / LEAST);
    const Cut cut{(int)max(1ll, min(pieces, (long long)MOST_CUT)), static_cast<float *>(c.pieces), static_cast<float *>(c.pieces) + (size_t)MOST_CTAS * 128 * kSlice,
                  c.jobs == 1 && c.job[0].first && c.job[0].first == c.job[0].last};
    const dim3 grid((unsigned)(c.N * c.H), wide, c.jobs);
    if (cut.pieces > 1) {
        scan_kernel<true><<<dim3(grid.x, grid.y, grid.z * (cut.pieces - 1)), THREADS, bytes, s>>>(c, cut);
        count_launch();
    }
    scan_kernel<false><<<dim3(grid.x, grid.y, grid.z * cut.pieces), THREADS, bytes, s>>>(c, cut);
    count_launch();
    return cudaGetLastError();
}

}  // namespace lin
}  // namespace k3kda
