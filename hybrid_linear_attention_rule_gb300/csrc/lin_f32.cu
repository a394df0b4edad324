// lin_f32.cu -- linear attention's jobs (lin.cuh) on the CUDA cores, everything in FP32: the path of FP32 inputs.
//
// A CTA holds a slice of 32 or 64 channels of one head's state [a, b] in shared memory and walks the sequence, or a piece of it, in chunks of 32 tokens, a token a
// lane for the decays; the next chunk's rows are on their way, in registers, meanwhile.  The four products of a chunk (x y^T, its
// product with z, x S, y^T z) are register tiles of 4 to 16 accumulators fed by 16-byte shared loads; the scores are worked out again by
// each slice of b.  What bounds it is the shared loads, some 5 for 16 products of a thread, and the sequence of its steps.
#include "lin.cuh"

namespace k3kda {
namespace lin {
namespace {

constexpr int C = 32, THREADS = 256, LEAST = 2;

struct Layout {
    int pa, x, y, z, s, p, w, total;       // floats
    __host__ __device__ Layout(int a, int width) {
        pa = a + 4;
        x = 0;
        y = x + C * pa;
        s = y + C * pa;
        z = s + a * (width + 4);
        p = z + C * (width + 4);
        w = p + C * (C + 1);
        total = w + 5 * C;
    }
};

// Pieces of each sequence, where there are fewer CTAs than the GPU holds: their states come from a first pass (STATES), which takes those
// of every piece but the last from zero, and a piece's own chain of those before it.
struct Cut {
    int pieces;
    float *state, *keep;       // [jobs][pieces][N H][slices] of [a, W] and of one; the last piece's holds the first state where it is written over
    bool kept;
};

template <bool STATES, int W> __global__ void __launch_bounds__(THREADS, 2) scan_kernel(const __grid_constant__ Call A, const Cut cut) {
    constexpr int PITCH_S = W + 4, ACROSS = W / 4, TOK = W / 32, ROWS = W / 8, STEP = THREADS / ACROSS;     // tiles of 4 channels: TOK tokens of outputs, ROWS rows of the state
    extern __shared__ float4 smem4[];
    __shared__ unsigned lost;              // tokens of the chunk whose decay is NaN
    const int parts = STATES ? cut.pieces - 1 : cut.pieces, job = blockIdx.z / parts, piece = blockIdx.z % parts;
    const Job &J = A.job[job];
    const int b0 = blockIdx.y * W, a = J.a, nb = min(W, J.b - b0);
    if (b0 >= J.b) return;
    float *sm = reinterpret_cast<float *>(smem4);
    const Layout L(a, W);
    float *X = sm + L.x, *Y = sm + L.y, *Z = sm + L.z, *S = sm + L.s, *P = sm + L.p;
    float *hi = sm + L.w, *lo = hi + C, *cin = lo + C, *wt = cin + C, *keep = wt + C;
    const int tid = threadIdx.x, n = blockIdx.x / A.H, h = blockIdx.x % A.H;
    int begin, end;
    seq_bounds(A.cu, n, A.T, begin, end);
    const int len = end - begin, chunks = (len + C - 1) / C;
    const int slot = seq_slot(A.slot, A.num_slots, n);
    const size_t state = ((size_t)(slot < 0 ? 0 : slot) * A.H + h) * a * J.b;
    const int tx = tid % ACROSS, ty = tid / ACROSS;

    const int begins = (int)((long long)chunks * piece / cut.pieces), ends = (int)((long long)chunks * (piece + 1) / cut.pieces);
    // a piece's place among the states
    auto place = [&](int p) { return (((size_t)job * cut.pieces + p) * gridDim.x + blockIdx.x) * gridDim.y + blockIdx.y; };
    long long units = 0;                   // STATES: the piece's decay (warp 0)
    unsigned gone = 0;
    if (piece == 0) {
        const float *kept = !STATES && cut.kept && cut.pieces > 1 ? cut.state + place(cut.pieces - 1) * (128 * W) : nullptr;
        for (int i = tid; i < a * W; i += THREADS) {
            const int c = i / W, b = i % W;
            const float v = kept ? kept[i] : J.first && slot >= 0 && b < nb ? J.first[state + (size_t)c * J.sa + (size_t)(b0 + b) * J.sb] : 0.f;
            S[c * PITCH_S + b] = v;
            if (STATES && cut.kept) cut.state[place(cut.pieces - 1) * (128 * W) + i] = v;
        }
    } else {
        float v[128 * W / THREADS];
#pragma unroll
        for (int k = 0; k < 128 * W / THREADS; ++k) v[k] = 0.f;
        if (!STATES)
            for (int p = 0; p < piece; ++p) {
                const float *from = cut.state + place(p) * (128 * W);
                const float e = cut.keep[place(p)];
#pragma unroll
                for (int k = 0; k < 128 * W / THREADS; ++k)
                    if (tid + k * THREADS < a * W) v[k] = fmaf(e, v[k], from[tid + k * THREADS]);
            }
#pragma unroll
        for (int k = 0; k < 128 * W / THREADS; ++k) {
            const int i = tid + k * THREADS;
            if (i < a * W) S[i / W * PITCH_S + i % W] = v[k];
        }
    }
    const size_t base_x = h / J.x.share, base_y = h / J.y.share, base_z = h / J.z.share;
    const size_t hx = A.H / J.x.share, hy = A.H / J.y.share, hz = A.H / J.z.share;

    // A chunk's rows as 16-byte pieces: piece i of x and y is row i / (a / 4), 4 pieces a thread at most; of z rows ty, ty + STEP.
    constexpr int MOST = C * 128 / 4 / THREADS;
    const int per_row = a / 4, pieces = C * per_row;
    float4 nx[MOST], ny[MOST], nz[TOK];
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
#pragma unroll
        for (int k = 0; k < TOK; ++k) {
            const int t = ty + k * STEP;
            nz[k] = t < valid && 4 * tx < nb ? *reinterpret_cast<const float4 *>(pz + ((size_t)(t0 + t) * hz + base_z) * J.b + b0 + 4 * tx) : none;
        }
        if (tid < C) ng = tid < valid ? A.g[A.fixed ? h : (size_t)(t0 + tid) * A.H + h] : 0.f;
    };
    if (begins < ends) fetch(begins);
    for (int it = begins; it < ends; ++it) {
        const int chunk = J.reverse ? chunks - 1 - it : it, t0 = begin + chunk * C, valid = min(C, end - t0);
        __syncthreads();
        if (!STATES && J.anchors && !J.reverse && it > 0 && chunk * C % kAnchor == 0) {
            float *to = J.anchors + ((size_t)(anchor_slot(begin, n) + chunk * C / kAnchor - 1) * A.H + h) * a * J.b;
            for (int i = tid; i < a * W; i += THREADS)
                if (i % W < nb) to[(size_t)(i / W) * J.b + b0 + i % W] = S[i / W * PITCH_S + i % W];
        }
#pragma unroll
        for (int k = 0; k < MOST; ++k) {
            const int i = tid + k * THREADS;
            if (i < pieces) {
                if (!STATES) *reinterpret_cast<float4 *>(X + i / per_row * L.pa + i % per_row * 4) = nx[k];
                *reinterpret_cast<float4 *>(Y + i / per_row * L.pa + i % per_row * 4) = ny[k];
            }
        }
#pragma unroll
        for (int k = 0; k < TOK; ++k) *reinterpret_cast<float4 *>(Z + (ty + k * STEP) * PITCH_S + 4 * tx) = nz[k];
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
                units = add_units(units, all);
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

        {   // outputs: tokens ty, ty + STEP, channels 4 tx .. 4 tx + 3
            float o[TOK][4] = {};
            for (int c = 0; c < a; c += 4) {
                float4 x[TOK];
#pragma unroll
                for (int k = 0; k < TOK; ++k) x[k] = *reinterpret_cast<float4 *>(X + (ty + k * STEP) * L.pa + c);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float4 v = *reinterpret_cast<float4 *>(S + (c + u) * PITCH_S + 4 * tx);
#pragma unroll
                    for (int k = 0; k < TOK; ++k) {
                        const float xc = u == 0 ? x[k].x : u == 1 ? x[k].y : u == 2 ? x[k].z : x[k].w;
                        o[k][0] = fmaf(xc, v.x, o[k][0]);
                        o[k][1] = fmaf(xc, v.y, o[k][1]);
                        o[k][2] = fmaf(xc, v.z, o[k][2]);
                        o[k][3] = fmaf(xc, v.w, o[k][3]);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < TOK; ++k) {
                const float ci = cin[ty + k * STEP];
#pragma unroll
                for (int u = 0; u < 4; ++u) o[k][u] *= ci;
            }
            // (a z that is not seen is left out, not multiplied by 0: it may be infinite)
            for (int j = 0; j < C; ++j) {
                const float4 z = *reinterpret_cast<float4 *>(Z + j * PITCH_S + 4 * tx);
#pragma unroll
                for (int k = 0; k < TOK; ++k) {
                    const int t = ty + k * STEP;
                    if (J.reverse ? j <= t : j >= t) continue;
                    const float p = P[t * (C + 1) + j];
                    o[k][0] = fmaf(p, z.x, o[k][0]);
                    o[k][1] = fmaf(p, z.y, o[k][1]);
                    o[k][2] = fmaf(p, z.z, o[k][2]);
                    o[k][3] = fmaf(p, z.w, o[k][3]);
                }
            }
#pragma unroll
            for (int k = 0; k < TOK; ++k) {
                const int t = ty + k * STEP;
                const size_t row = (size_t)(t0 + t) * A.H + h;
                if (J.dots) {
                    float dot = 0.f;
                    if (t < valid)
                        for (int u = 0; u < 4; ++u)
                            if (4 * tx + u < nb)
                                dot = fmaf(load_elt(J.r.p, ((size_t)(t0 + t) * (A.H / J.r.share) + h / J.r.share) * J.b + b0 + 4 * tx + u, 0), o[k][u], dot);
#pragma unroll
                    for (int u = 1; u < ACROSS; u <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, u);
                    if (t < valid && tx == 0) J.dots[(size_t)blockIdx.y * A.T * A.H + row] = dot;
                }
                if (t < valid) {
                    const float p = P[t * (C + 1) + t];
                    for (int u = 0; u < 4; ++u)
                        if (4 * tx + u < nb) store_elt(J.out, row * J.b + b0 + 4 * tx + u, fmaf(p, Z[t * PITCH_S + 4 * tx + u], o[k][u]), J.out_bf16);
                }
            }
        }
        __syncthreads();
        }

        // the state: rows ROWS ty and on, channels 4 tx .. 4 tx + 3
        if (ROWS * ty < a) {
            float acc[ROWS][4];
            const float e = *keep;
#pragma unroll
            for (int u = 0; u < ROWS; ++u) {
                const float4 v = *reinterpret_cast<float4 *>(S + (ROWS * ty + u) * PITCH_S + 4 * tx);
                acc[u][0] = e * v.x;
                acc[u][1] = e * v.y;
                acc[u][2] = e * v.z;
                acc[u][3] = e * v.w;
            }
            for (int j = 0; j < valid; ++j) {
                const float4 z = *reinterpret_cast<float4 *>(Z + j * PITCH_S + 4 * tx);
                const float w = wt[j];
#pragma unroll
                for (int r = 0; r < ROWS; r += 4) {
                    const float4 y = *reinterpret_cast<float4 *>(Y + j * L.pa + ROWS * ty + r);
                    const float yw[4] = {w * y.x, w * y.y, w * y.z, w * y.w};
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        acc[r + u][0] = fmaf(yw[u], z.x, acc[r + u][0]);
                        acc[r + u][1] = fmaf(yw[u], z.y, acc[r + u][1]);
                        acc[r + u][2] = fmaf(yw[u], z.z, acc[r + u][2]);
                        acc[r + u][3] = fmaf(yw[u], z.w, acc[r + u][3]);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < ROWS; ++u)
                *reinterpret_cast<float4 *>(S + (ROWS * ty + u) * PITCH_S + 4 * tx) = make_float4(acc[u][0], acc[u][1], acc[u][2], acc[u][3]);
        }
        if (!STATES && J.anchors && J.reverse && chunk > 0 && chunk * C % kAnchor == 0) {
            __syncthreads();
            float *to = J.anchors + ((size_t)(anchor_slot(begin, n) + chunk * C / kAnchor - 1) * A.H + h) * a * J.b;
            for (int i = tid; i < a * W; i += THREADS)
                if (i % W < nb) to[(size_t)(i / W) * J.b + b0 + i % W] = S[i / W * PITCH_S + i % W];
        }
    }
    __syncthreads();
    if (STATES) {
        for (int i = tid; i < a * W; i += THREADS) cut.state[place(piece) * (128 * W) + i] = S[i / W * PITCH_S + i % W];
        if (tid == 0) cut.keep[place(piece)] = gone ? __int_as_float(0x7fffffff) : exp2_units(units);
        return;
    }
    if (piece < cut.pieces - 1) return;
    for (int i = tid; i < a * W; i += THREADS) {
        const int c = i / W, b = i % W;
        if (b >= nb) continue;
        const float v = S[c * PITCH_S + b];
        if (J.last && slot >= 0) J.last[state + (size_t)c * J.sa + (size_t)(b0 + b) * J.sb] = v;
        if (J.anchors && J.last_anchor)
            J.anchors[((size_t)(anchor_slot(begin, n) + max(0, len - 1) / kAnchor) * A.H + h) * a * J.b + (size_t)c * J.b + b0 + b] = v;
    }
}

std::atomic<uint64_t> g_attr[4];

constexpr int MOST_CTAS = 320, MOST_CUT = 64;

template <int W> cudaError_t launch(const Call &c, std::atomic<uint64_t> *attr, cudaStream_t s) {
    const int most = (int)(Layout(128, W).total * sizeof(float));
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = smem_attr_once((const void *)scan_kernel<false, W>, most, attr[0]);
    if (e == cudaSuccess) e = smem_attr_once((const void *)scan_kernel<true, W>, most, attr[1]);
    if (e != cudaSuccess) return e;
    int wide = 0, bytes = 0;
    for (int j = 0; j < c.jobs; ++j) {
        wide = max(wide, (c.job[j].b + W - 1) / W);
        bytes = max(bytes, (int)(Layout(c.job[j].a, W).total * sizeof(float)));
    }
    // Two CTAs an SM, pieces of LEAST chunks or more on average.  (Slices of 32 channels, heads of 128, uncut and cut: 8 heads of 8,192 tokens 1,938 and
    // 479 us, of 1,024 tokens 247 and 79, of 256 tokens 67 and 34, where pieces of 4 chunks took 50; 32 heads of 2,048 tokens 492 and 495; gradients
    // of 8 heads of 8,192 tokens 2,279 and 1,513.  Three or four CTAs an SM in turn were no faster.)
    const long long ctas = (long long)c.N * c.H * wide * c.jobs, chunks = c.T / C / c.N;
    long long pieces = min((long long)min(2 * sms, MOST_CTAS) / ctas, chunks / LEAST);
    const Cut cut{(int)max(1ll, min(pieces, (long long)MOST_CUT)), static_cast<float *>(c.pieces), static_cast<float *>(c.pieces) + (size_t)MOST_CTAS * 128 * W,
                  c.jobs == 1 && c.job[0].first && c.job[0].first == c.job[0].last};
    const dim3 grid((unsigned)(c.N * c.H), wide, c.jobs);
    if (cut.pieces > 1) {
        scan_kernel<true, W><<<dim3(grid.x, grid.y, grid.z * (cut.pieces - 1)), THREADS, bytes, s>>>(c, cut);
        if ((e = launched()) != cudaSuccess) return e;
    }
    scan_kernel<false, W><<<dim3(grid.x, grid.y, grid.z * cut.pieces), THREADS, bytes, s>>>(c, cut);
    return launched();
}

}  // namespace

size_t f32_workspace() { return (size_t)MOST_CTAS * (128 * 64 + 1) * sizeof(float); }

cudaError_t launch_scan_f32(const Call &c, cudaStream_t s) {
    if (c.N == 0) return cudaSuccess;
    int b = 0;
    for (int j = 0; j < c.jobs; ++j) b = max(b, c.job[j].b);
    return slice_width(c.N, c.T, c.H, c.jobs, b) == 64 ? launch<64>(c, g_attr, s) : launch<32>(c, g_attr + 2, s);
}

}  // namespace lin
}  // namespace k3kda
