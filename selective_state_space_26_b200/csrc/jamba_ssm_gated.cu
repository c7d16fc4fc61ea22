// jamba_ssm_gated.cu -- host side of the C ABI declared in
// include/jamba_ssm_gated.h: argument validation and the launches of the gated
// recurrence's kernels.  Built as its own library, so its kernels and status
// word form a module of their own.  Nothing here allocates device memory.
#include "jamba_ssm_gated.h"

#include "gated_scan.cuh"
#include "gated_scan_bwd.cuh"
#include "gated_update.cuh"
#include "host_utils.h"

#define JSSM_GATED_API extern "C" __attribute__((visibility("default")))

using namespace jssm_host;

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 30, kMaxBatch = int64_t(1) << 24,
                  kMaxWidth = int64_t(1) << 20;

// Bytes from a strided activation's first element to its last one's end.
size_t span(int64_t rows, int64_t stride, int64_t d, int es) {
    return rows > 0 ? size_t((rows - 1) * stride + d) * es : 0;
}

// What the scan and its backward check alike.  Resolves the strides of 0.
template <typename P> jamba_ssm_status check_common(P *p, int64_t *rows) {
    if (p->batch < 0 || p->seqlen < 0 || p->d_inner < 1 || p->reserved != 0)
        return JAMBA_SSM_ERR_INVALID_ARG;
    if (p->io_dtype != JAMBA_SSM_BF16 && p->io_dtype != JAMBA_SSM_F32) return JAMBA_SSM_ERR_INVALID_ARG;
    if (p->cu_seqlens && p->total_tokens < 0) return JAMBA_SSM_ERR_INVALID_ARG;
    for (int64_t *s : {&p->x_stride, &p->g_stride, &p->z_stride}) {
        if (*s == 0) *s = p->d_inner;
        if (*s < p->d_inner) return JAMBA_SSM_ERR_INVALID_ARG;
        if (*s > (int64_t(1) << 31)) return JAMBA_SSM_ERR_UNSUPPORTED;
    }
    if (p->batch > kMaxBatch || p->d_inner > kMaxWidth || p->seqlen > kMaxRows)
        return JAMBA_SSM_ERR_UNSUPPORTED;
    *rows = p->cu_seqlens ? p->total_tokens : p->batch * p->seqlen;
    if (*rows > kMaxRows) return JAMBA_SSM_ERR_UNSUPPORTED;
    if (!aligned(p->cu_seqlens, 4) || !aligned(p->rate, 4) || !aligned(p->bias, 4) ||
        !aligned(p->h0, 4))
        return JAMBA_SSM_ERR_MISALIGNED;
    const int es = p->io_dtype == JAMBA_SSM_BF16 ? 2 : 4;
    if (!aligned(p->x, es) || !aligned(p->g, es) || !aligned(p->z, es)) return JAMBA_SSM_ERR_MISALIGNED;
    return JAMBA_SSM_OK;
}

template <typename P> void fill_common(const P &p, int64_t rows, jssm::GatedArgs *a) {
    a->x = p.x;
    a->g = p.g;
    a->z = p.z;
    a->xs = p.x_stride;
    a->gs = p.g_stride;
    a->zs = p.z_stride;
    a->rate = p.rate;
    a->bias = p.bias;
    a->h0 = p.h0;
    a->cu = p.cu_seqlens;
    a->total = rows;
    a->seqlen = p.seqlen;
    a->d = static_cast<int>(p.d_inner);
    a->batch = static_cast<int>(p.batch);
}

// How the rows can be read: bytes of one copy, the largest of 16, 4 and 2 that
// divides the width, the strides and every pointer.
int copy_bytes(const jssm::GatedArgs &a, int32_t dtype) {
    const int es = dtype == JAMBA_SSM_BF16 ? 2 : 4;
    int64_t bits = int64_t(a.d) * es;
    for (int64_t s : {a.xs, a.gs, a.zs}) bits |= s * es;
    for (const void *p : {a.x, a.g, a.z, (const void *)a.out, a.dout, (const void *)a.dx,
                          (const void *)a.dg, (const void *)a.dz})
        bits |= static_cast<int64_t>(reinterpret_cast<uintptr_t>(p));
    return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 2;
}

// How the work is cut: q runs side by side in a warp, cs CTAs in a cluster.
struct Cut {
    int q, cs;
    int64_t units;  // clusters
};

// Of a pass over sequences of tiles(q) channel tiles each.  A CTA of q = 1 reads 128 bytes of a row and takes 64 rows a round;
// q = 2 and 4 halve and quarter the width for two and four times the rows.
// Measured on 148 SMs (bf16 with z, us; before the maps held P - 1, which takes
// about 3% more on every side):
//   8192 channels, 4096 rows:  q 1 89, q 2 59, q 4 72, q 2 in clusters of 2 68;
//   2048 channels, 65536 rows: q 2 in clusters of 8 264, of 4 378, q 4 of 4 303;
//   512 channels, 8192 rows:   q 4 in clusters of 8 17, q 2 of 8 26, q 1 of 8 37;
//   13 x 4096 rows x 2048:     q 1 158, q 2 165, in clusters of 8 from 247.
// So: one CTA to a tile where 2 (q = 1) or 1.5 (q = 2) of them come to an SM;
// else clusters, whose barrier costs about a round's time and is hidden by the
// other CTAs of an SM, up to the per_sm that fit one (4 of the scan's, 2 of the
// backward's); q = 4 where that leaves under half of them.  The backward alike: 1024
// channels, 4096 rows, both passes: q 2 in clusters of 8 39, q 4 of 4 44, of 8 50.
// Packed sequences are ragged: the longest, taken as three times the mean, may
// run on alone, so q goes up until its rounds take no longer than moving all
// the bytes (9 sequences, 3001 rows of 1000 fp32 channels, both passes: q 1 112,
// q 2 66, q 4 52; 33 sequences, 16384 rows of 4096: q 1 94, q 2 113, q 4 160).
// The host does not know the lengths.  Where one is far longer than that, it does
// run on alone: 8192 rows and 255 of one row, 4096 channels, 219 us, 357 with the
// long one last (more sequences than a CTA has threads keep their order), for 70 of
// the long one by itself.
struct Pass {
    int per_sm, per_sm4;  // CTAs that fit an SM, and of q = 4
    int halves;           // half CTAs to an SM from which q = 2 takes no cluster
    double round_us;  // a round of one CTA
    int arrays;       // activations read and written
};
template <typename Tiles>
Cut choose_cut(const jssm::GatedArgs &a, int es, int sms, const Pass &pass, Tiles tiles) {
    const int64_t batch = a.batch, len = a.cu ? a.total / batch : a.seqlen;
    auto clusters = [&](int q) {
        const int64_t units = batch * tiles(q), rows = int64_t(jssm::kGatedCkpt) * q;
        int cs = 1;
        while (cs < jssm::kGatedMaxCluster && cs * 2 <= (len + rows - 1) / rows &&
               units * cs * 2 <= int64_t(q == 4 ? pass.per_sm4 : pass.per_sm) * sms)
            cs *= 2;
        return Cut{q, cs, units};
    };
    const bool ragged = a.cu && batch > 1;
    const double all_us = double(a.total) * a.d * es * pass.arrays / 5.2e6;
    auto alone_ok = [&](int q) {
        return !ragged || 3.0 * len / (jssm::kGatedCkpt * q) * pass.round_us <= all_us;
    };
    if (batch * tiles(1) >= 2 * sms && alone_ok(1)) return {1, 1, batch * tiles(1)};
    if (batch * tiles(2) * 2 >= pass.halves * sms) {
        const int q = alone_ok(2) ? 2 : 4;
        return {q, 1, batch * tiles(q)};
    }
    const Cut two = clusters(2);
    return two.units * two.cs * 2 < int64_t(pass.per_sm4) * sms ? clusters(4) : two;
}

using Bf = __nv_bfloat16;

struct Kernel {
    const void *fn;
    int threads, smem;
};

// Raises a kernel's dynamic shared-memory limit, once per kernel and device.
cudaError_t raise_smem(const Kernel &k, int dev) {
    static std::mutex mutex;
    static const void *done[kMaxDevices][128];
    std::lock_guard<std::mutex> lock(mutex);
    for (const void *&slot : done[dev]) {
        if (slot == k.fn) return cudaSuccess;
        if (slot == nullptr) {
            const cudaError_t e =
                cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
            if (e == cudaSuccess) slot = k.fn;
            return e;
        }
    }
    return cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
}

jamba_ssm_status launch_clusters(const Kernel &k, int64_t units, int cs, void **args,
                                 const DeviceInfo *dev, void *stream) {
    if (units * cs > 0x7fffffff) return JAMBA_SSM_ERR_UNSUPPORTED;
    const cudaError_t e = raise_smem(k, dev->id);
    if (e != cudaSuccess) return cuda_fail(e);
    // not early: CTAs that wait beside the kernel before them take the free SMs'
    // room first, and the cut's even share of the device is lost (220 us for 189)
    return launch(k.fn, dim3(static_cast<unsigned>(units * cs)), unsigned(k.threads), k.smem, cs, false,
                  args, stream);
}

template <typename T, int VEC, int CP, int Q, bool CL, int W> Kernel scan_kernel_w(bool gate) {
    using G = jssm::GatedScanCfg<true, W, Q, CP>;
    using N = jssm::GatedScanCfg<false, W, Q, CP>;
    if constexpr (CP == jssm::kCpShifted)  // with z only
        return Kernel{(const void *)&jssm::gated_scan_kernel<T, VEC, true, Q, CP, CL, W>, G::kThreads,
                      G::kSmemBytes};
    else
        return gate ? Kernel{(const void *)&jssm::gated_scan_kernel<T, VEC, true, Q, CP, CL, W>, G::kThreads,
                             G::kSmemBytes}
                    : Kernel{(const void *)&jssm::gated_scan_kernel<T, VEC, false, Q, CP, CL, W>, N::kThreads,
                             N::kSmemBytes};
}
template <typename T, int VEC, int CP, bool CL> Kernel scan_kernel_q(bool gate, int q) {
    return q == 1 ? scan_kernel_w<T, VEC, CP, 1, CL, 4>(gate)
         : q == 2 ? scan_kernel_w<T, VEC, CP, 2, CL, 4>(gate)
                  : scan_kernel_w<T, VEC, CP, 4, CL, 4>(gate);
}
template <typename T, int VEC, int CP> Kernel scan_kernel(bool gate, const Cut &cut, int sms) {
    // Two of 8 warps fit an SM as four of 4 do, and take half the rounds: 8192
    // channels, 4096 rows 57 us for 61.  Not for fp32, whose rows are as long in
    // bytes at half the channels (4096 x 4096: 48 for 44), nor where more than two
    // CTAs come to an SM (13 x 4096 x 2048: 177 for 170), nor for the shifted
    // copies, whose stages leave room for one of 8 warps and three of 4 (4096 x
    // 8194 110 for 100, 24 x 300 x 310 15.9 for 12.3).
    if constexpr (VEC == 2 && CP != jssm::kCpShifted)
        if (cut.cs == 1 && cut.q == 2 && cut.units <= 2 * sms) return scan_kernel_w<T, VEC, CP, 2, false, 8>(gate);
    if constexpr (VEC == 2 && CP == jssm::kCpShifted)  // without a cluster only
        return scan_kernel_q<T, VEC, CP, false>(gate, cut.q);
    else
        return cut.cs > 1 ? scan_kernel_q<T, VEC, CP, true>(gate, cut.q) : scan_kernel_q<T, VEC, CP, false>(gate, cut.q);
}

jamba_ssm_status launch_scan(jssm::GatedArgs &a, int32_t dtype, const DeviceInfo *dev, void *stream) {
    const int cp = copy_bytes(a, dtype);
    const bool bf = dtype == JAMBA_SSM_BF16, gate = a.z != nullptr;
    const int width = bf && cp >= 4 ? 64 : 32;  // channels of a warp's row
    // Rows that begin at any multiple of 4 bytes, where three arrays are read: 16-byte
    // copies of what holds them (us, 4-byte copies first: fp32 8 x 2048 x 4099 305
    // and 231, 8192 x 515 43 and 28, 50001 x 1001 394 and 297; bf16 13 x 4096 x 1026
    // 184 and 135).  Not for two arrays (50001 x 1001 fp32 182 and 195; 8192 x 514
    // bf16 14 and 17) nor for bf16 in clusters (8192 x 2050 66 and 89).  Their stages
    // are larger: three CTAs fit an SM, two of q = 4, and a cluster's barrier is
    // hidden by fewer (8192 x 2501 x 2 fp32, q 2: one CTA to a tile 88, clusters of 4
    // 120; 20001 x 1601: clusters of 2 233, of 4 158, of 8 209).
    const bool any4 = cp == 4 && gate && aligned(a.x, 16) && aligned(a.g, 16) && aligned(a.z, 16);
    const Pass pass = any4 && !bf ? Pass{3, 2, 2, 1.4, 4} : Pass{4, 4, 3, 1.4, gate ? 4 : 3};
    const Cut cut = choose_cut(a, bf ? 2 : 4, dev->sms, pass,
                               [&](int q) { return int64_t(a.d + width / q - 1) / (width / q); });
    const bool shifted = any4 && (!bf || cut.cs == 1);
    int cs = cut.cs;
    void *args[] = {&a, &cs};
    const Kernel k = !bf ? (cp == 16 ? scan_kernel<float, 1, 16>(gate, cut, dev->sms)
                            : shifted ? scan_kernel<float, 1, jssm::kCpShifted>(gate, cut, dev->sms)
                                      : scan_kernel<float, 1, 4>(gate, cut, dev->sms))
                     : cp == 16 ? scan_kernel<Bf, 2, 16>(gate, cut, dev->sms)
                     : shifted  ? scan_kernel<Bf, 2, jssm::kCpShifted>(gate, cut, dev->sms)
                     : cp == 4  ? scan_kernel<Bf, 2, 4>(gate, cut, dev->sms)
                                : scan_kernel<Bf, 1, 2>(gate, cut, dev->sms);
    return launch_clusters(k, cut.units, cs, args, dev, stream);
}

template <typename T, int VEC, int CP, int Q, bool CL> Kernel bwd_kernel_q(bool gate) {
    return gate ? Kernel{(const void *)&jssm::gated_scan_bwd_kernel<T, VEC, true, Q, CP, CL>,
                         jssm::kGatedBwdThreads, jssm::GatedBwdCfg<true>::kSmemBytes}
                : Kernel{(const void *)&jssm::gated_scan_bwd_kernel<T, VEC, false, Q, CP, CL>,
                         jssm::kGatedBwdThreads, jssm::GatedBwdCfg<false>::kSmemBytes};
}
template <typename T, int VEC, int CP, bool CL> Kernel bwd_kernel_c(bool gate, int q) {
    return q == 1 ? bwd_kernel_q<T, VEC, CP, 1, CL>(gate)
         : q == 2 ? bwd_kernel_q<T, VEC, CP, 2, CL>(gate)
                  : bwd_kernel_q<T, VEC, CP, 4, CL>(gate);
}
template <typename T, int VEC, int CP> Kernel bwd_kernel(bool gate, int q, int cs) {
    return cs > 1 ? bwd_kernel_c<T, VEC, CP, true>(gate, q) : bwd_kernel_c<T, VEC, CP, false>(gate, q);
}

jamba_ssm_status launch_bwd(jssm::GatedArgs &a, int32_t dtype, const DeviceInfo *dev, void *stream) {
    const int cp = copy_bytes(a, dtype);
    const bool bf = dtype == JAMBA_SSM_BF16, gate = a.z != nullptr;
    const int width = bf && cp >= 4 ? 64 : 32;
    const Cut cut = choose_cut(a, bf ? 2 : 4, dev->sms, Pass{2, 2, 3, 2.4, gate ? 7 : 5},
                               [&](int q) { return int64_t(a.d + width / q - 1) / (width / q); });
    int q = cut.q, cs = cut.cs;
    void *args[] = {&a, &cs};
    const Kernel k = !bf ? (cp == 16 ? bwd_kernel<float, 1, 16>(gate, q, cs) : bwd_kernel<float, 1, 4>(gate, q, cs))
                     : cp == 16 ? bwd_kernel<Bf, 2, 16>(gate, q, cs)
                     : cp == 4  ? bwd_kernel<Bf, 2, 4>(gate, q, cs)
                                : bwd_kernel<Bf, 1, 2>(gate, q, cs);
    return launch_clusters(k, cut.units, cs, args, dev, stream);
}

size_t ckpt_bytes(int64_t batch, int64_t rows, int64_t d) {
    return size_t(rows / JAMBA_SSM_GATED_CKPT_STEPS + batch) * size_t(d) * 4;
}
size_t partial_bytes(int64_t batch, int64_t d) { return size_t(batch) * 2 * size_t(d) * 4; }

}  // namespace

JSSM_GATED_API size_t jamba_ssm_gated_scan_ckpt_size(int64_t batch, int64_t rows, int64_t d_inner) {
    return batch < 0 || rows < 0 || d_inner < 0 ? 0 : ckpt_bytes(batch, rows, d_inner);
}

JSSM_GATED_API size_t jamba_ssm_gated_scan_bwd_workspace_size(int64_t batch, int64_t rows,
                                                              int64_t d_inner, int32_t has_ckpt) {
    if (batch < 0 || rows < 0 || d_inner < 0) return 0;
    return partial_bytes(batch, d_inner) + (has_ckpt ? 0 : ckpt_bytes(batch, rows, d_inner));
}

JSSM_GATED_API jamba_ssm_status jamba_ssm_gated_scan(const jamba_ssm_gated_scan_params *pin,
                                                     void *stream) {
    jamba_ssm_gated_scan_params p;
    if (!read_params(pin, &p)) return JAMBA_SSM_ERR_INVALID_ARG;
    int64_t rows = 0;
    jamba_ssm_status st = check_common(&p, &rows);
    if (st != JAMBA_SSM_OK) return st;
    if (p.initial_indices && !p.state_indices) return JAMBA_SSM_ERR_INVALID_ARG;
    if (p.state_indices && p.num_slots < 1) return JAMBA_SSM_ERR_INVALID_ARG;
    if (p.num_slots > 0x7fffffff) return JAMBA_SSM_ERR_UNSUPPORTED;
    const int es = p.io_dtype == JAMBA_SSM_BF16 ? 2 : 4;
    if (!aligned(p.state_indices, 4) || !aligned(p.initial_indices, 4) || !aligned(p.out, es) ||
        !aligned(p.h_final, 4) || !aligned(p.ckpt, 16))
        return JAMBA_SSM_ERR_MISALIGNED;
    if ((st = check_workspace(p.workspace, p.workspace_bytes)) != JAMBA_SSM_OK) return st;
    if (p.batch == 0) return JAMBA_SSM_OK;  // no work; the pointers are not used
    if (rows > 0 && (!p.x || !p.g || !p.out)) return JAMBA_SSM_ERR_INVALID_ARG;
    const size_t act = size_t(rows) * p.d_inner * es;
    const size_t state = size_t(p.state_indices ? p.num_slots : p.batch) * p.d_inner * 4;
    const Range ins[] = {{p.x, span(rows, p.x_stride, p.d_inner, es)},
                         {p.g, span(rows, p.g_stride, p.d_inner, es)},
                         {p.z, span(rows, p.z_stride, p.d_inner, es)},
                         {p.rate, size_t(p.d_inner) * 4},
                         {p.bias, size_t(p.d_inner) * 4},
                         {p.cu_seqlens, size_t(p.batch + 1) * 4},
                         {p.state_indices, size_t(p.batch) * 4},
                         {p.initial_indices, size_t(p.batch) * 4},
                         {p.h0 == p.h_final ? nullptr : p.h0, state}};
    const Range outs[] = {{p.out, act},
                          {p.h_final, state},
                          {p.ckpt, ckpt_bytes(p.batch, rows, p.d_inner)},
                          {p.workspace, size_t(JAMBA_SSM_STATUS_BYTES)}};
    if (any_overlap(outs, 4, ins, 9)) return JAMBA_SSM_ERR_INVALID_ARG;
    const DeviceInfo *dev = current_device(&st);
    if (!dev) return st;

    jssm::GatedArgs a{};
    fill_common(p, rows, &a);
    a.out = p.out;
    a.h_final = p.h_final;
    a.state_indices = p.state_indices;
    a.initial_indices = p.initial_indices;
    a.num_slots = p.num_slots;
    a.ckpt = p.ckpt;
    a.status = static_cast<int *>(p.workspace);
    if ((st = launch_scan(a, p.io_dtype, dev, stream)) != JAMBA_SSM_OK) return st;
    return finish_launch(stream, p.workspace);
}

JSSM_GATED_API jamba_ssm_status
jamba_ssm_gated_scan_bwd(const jamba_ssm_gated_scan_bwd_params *pin, void *stream) {
    jamba_ssm_gated_scan_bwd_params p;
    if (!read_params(pin, &p)) return JAMBA_SSM_ERR_INVALID_ARG;
    int64_t rows = 0;
    jamba_ssm_status st = check_common(&p, &rows);
    if (st != JAMBA_SSM_OK) return st;
    const int es = p.io_dtype == JAMBA_SSM_BF16 ? 2 : 4;
    if (!aligned(p.dout, es) || !aligned(p.dx, es) || !aligned(p.dg, es) || !aligned(p.dz, es) ||
        !aligned(p.dh_final, 4) || !aligned(p.drate, 4) || !aligned(p.dbias, 4) ||
        !aligned(p.dh0, 4) || !aligned(p.ckpt, 16) || !aligned(p.workspace, 16))
        return JAMBA_SSM_ERR_MISALIGNED;
    const size_t need = jamba_ssm_gated_scan_bwd_workspace_size(p.batch, rows, p.d_inner, p.ckpt != nullptr);
    if (need > 0 && (!p.workspace || p.workspace_bytes < need)) return JAMBA_SSM_ERR_WORKSPACE;
    if (rows > 0 && p.batch > 0 &&
        (!p.x || !p.g || !p.dout || !p.dx || !p.dg || (p.z != nullptr) != (p.dz != nullptr)))
        return JAMBA_SSM_ERR_INVALID_ARG;
    const size_t act = size_t(rows) * p.d_inner * es, state = size_t(p.batch) * p.d_inner * 4;
    const size_t par = size_t(p.d_inner) * 4;
    const Range ins[] = {{p.x, span(rows, p.x_stride, p.d_inner, es)},
                         {p.g, span(rows, p.g_stride, p.d_inner, es)},
                         {p.z, span(rows, p.z_stride, p.d_inner, es)},
                         {p.rate, par},
                         {p.bias, par},
                         {p.cu_seqlens, size_t(p.batch + 1) * 4},
                         {p.h0, state},
                         {p.dout, act},
                         {p.dh_final, state},
                         {p.ckpt, ckpt_bytes(p.batch, rows, p.d_inner)}};
    const Range outs[] = {{p.dx, act},   {p.dg, act},    {p.dz, act},   {p.drate, par},
                          {p.dbias, par}, {p.dh0, state}, {p.workspace, need}};
    if (any_overlap(outs, 7, ins, 10)) return JAMBA_SSM_ERR_INVALID_ARG;
    const DeviceInfo *dev = current_device(&st);
    if (!dev) return st;

    jssm::GatedArgs a{};
    fill_common(p, rows, &a);
    a.dout = p.dout;
    a.dh_final = p.dh_final;
    a.dx = p.dx;
    a.dg = p.dg;
    a.dz = p.dz;
    a.drate = p.drate;
    a.dbias = p.dbias;
    a.dh0 = p.dh0;
    a.partial = static_cast<float *>(p.workspace);
    a.ckpt = const_cast<float *>(p.ckpt);
    if (p.batch > 0) {
        if (!a.ckpt) {
            a.ckpt = a.partial + partial_bytes(p.batch, p.d_inner) / 4;
            if ((st = launch_scan(a, p.io_dtype, dev, stream)) != JAMBA_SSM_OK) return st;
        }
        if (p.batch == 1) a.partial = nullptr;  // one sequence's sums are the sums
        if ((st = launch_bwd(a, p.io_dtype, dev, stream)) != JAMBA_SSM_OK) return st;
    }
    if ((a.drate || a.dbias) && p.batch != 1) {
        void *args[] = {&a.partial, &a.drate, &a.dbias, &a.batch, &a.d};
        st = launch_early((const void *)&jssm::gated_reduce_kernel, dim3(unsigned((a.d + 127) / 128)), 128, 0, 1,
                          args, stream);
        if (st != JAMBA_SSM_OK) return st;
    }
    return finish_launch(stream, nullptr);
}

JSSM_GATED_API jamba_ssm_status
jamba_ssm_gated_state_update(const jamba_ssm_gated_state_update_params *pin, void *stream) {
    jamba_ssm_gated_state_update_params p;
    if (!read_params(pin, &p)) return JAMBA_SSM_ERR_INVALID_ARG;
    if (p.batch < 0 || p.d_inner < 1 || p.reserved != 0) return JAMBA_SSM_ERR_INVALID_ARG;
    if (p.io_dtype != JAMBA_SSM_BF16 && p.io_dtype != JAMBA_SSM_F32) return JAMBA_SSM_ERR_INVALID_ARG;
    if (p.state_indices && p.num_slots < 1) return JAMBA_SSM_ERR_INVALID_ARG;
    for (int64_t *s : {&p.x_stride, &p.g_stride, &p.z_stride}) {
        if (*s == 0) *s = p.d_inner;
        if (*s < p.d_inner) return JAMBA_SSM_ERR_INVALID_ARG;
        if (*s > (int64_t(1) << 31)) return JAMBA_SSM_ERR_UNSUPPORTED;
    }
    if (p.batch > kMaxBatch || p.d_inner > kMaxWidth || p.num_slots > 0x7fffffff)
        return JAMBA_SSM_ERR_UNSUPPORTED;
    const int es = p.io_dtype == JAMBA_SSM_BF16 ? 2 : 4;
    if (!aligned(p.x, es) || !aligned(p.g, es) || !aligned(p.z, es) || !aligned(p.out, es) ||
        !aligned(p.state, 4) || !aligned(p.rate, 4) || !aligned(p.bias, 4) || !aligned(p.state_indices, 4))
        return JAMBA_SSM_ERR_MISALIGNED;
    jamba_ssm_status st = check_workspace(p.workspace, p.workspace_bytes);
    if (st != JAMBA_SSM_OK) return st;
    if (p.batch == 0) return JAMBA_SSM_OK;
    if (!p.state || !p.x || !p.g || !p.out) return JAMBA_SSM_ERR_INVALID_ARG;
    const size_t state = size_t(p.state_indices ? p.num_slots : p.batch) * p.d_inner * 4;
    const Range ins[] = {{p.x, span(p.batch, p.x_stride, p.d_inner, es)},
                         {p.g, span(p.batch, p.g_stride, p.d_inner, es)},
                         {p.z, span(p.batch, p.z_stride, p.d_inner, es)},
                         {p.rate, size_t(p.d_inner) * 4},
                         {p.bias, size_t(p.d_inner) * 4},
                         {p.state_indices, size_t(p.batch) * 4}};
    const Range outs[] = {{p.out, size_t(p.batch) * p.d_inner * es},
                          {p.state, state},
                          {p.workspace, size_t(JAMBA_SSM_STATUS_BYTES)}};
    if (any_overlap(outs, 3, ins, 6)) return JAMBA_SSM_ERR_INVALID_ARG;
    if (!current_device(&st)) return st;

    jssm::GatedUpdateArgs a{};
    a.state = p.state;
    a.x = p.x;
    a.g = p.g;
    a.z = p.z;
    a.xs = p.x_stride;
    a.gs = p.g_stride;
    a.zs = p.z_stride;
    a.rate = p.rate;
    a.bias = p.bias;
    a.out = p.out;
    a.state_indices = p.state_indices;
    a.num_slots = p.num_slots;
    a.status = static_cast<int *>(p.workspace);
    a.d = static_cast<int>(p.d_inner);
    a.batch = static_cast<int>(p.batch);
    void *args[] = {&a};
    // 16-byte rows throughout: 8 bf16 or 4 fp32 channels a thread
    const int v = p.io_dtype == JAMBA_SSM_BF16 ? 8 : 4;
    bool wide = p.d_inner % v == 0;
    for (int64_t s : {p.x_stride, p.g_stride, p.z_stride}) wide = wide && s % v == 0;
    for (const void *q : {p.x, p.g, p.z, (const void *)p.out, (const void *)p.state,
                          (const void *)p.rate, (const void *)p.bias})
        wide = wide && aligned(q, 16);
    const void *k = p.io_dtype == JAMBA_SSM_BF16
                        ? (wide ? (const void *)&jssm::gated_update_kernel<Bf, 8>
                                : (const void *)&jssm::gated_update_kernel<Bf, 1>)
                        : (wide ? (const void *)&jssm::gated_update_kernel<float, 4>
                                : (const void *)&jssm::gated_update_kernel<float, 1>);
    const int64_t per = int64_t(jssm::kUpdateThreads) * (wide ? v : 1);
    const dim3 grid(static_cast<unsigned>((p.d_inner + per - 1) / per),
                    static_cast<unsigned>(p.batch < 65535 ? p.batch : 65535));
    st = launch_early(k, grid, jssm::kUpdateThreads, 0, 1, args, stream);
    if (st != JAMBA_SSM_OK) return st;
    return finish_launch(stream, p.workspace);
}

JSSM_GATED_API jamba_ssm_status jamba_ssm_gated_get_status(void *workspace, void *stream) {
    return read_status(workspace, stream);
}
JSSM_GATED_API int jamba_ssm_gated_last_cuda_error(void) { return t_last_cuda_error; }
JSSM_GATED_API int jamba_ssm_gated_abi_version(void) { return JAMBA_SSM_GATED_ABI_VERSION; }
