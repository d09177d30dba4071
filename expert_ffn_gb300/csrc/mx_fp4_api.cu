// mx_fp4_api.cu -- the microscaled 4-bit entry points of include/mx_moe.h: argument
// validation (all of it on the host, before any CUDA call) and the choice of tile, split
// and grid for each launch.
#include "mx_fp4.cuh"
#include "mx_fp4_choice.h"
#include "mx_host.h"

#include <algorithm>

using namespace mx;
using namespace mx::fp4;

namespace {

constexpr int kMaxCols = 1 << 20, kMaxRows = 1 << 28;
constexpr int kSmem = 227 * 1024;  // shared memory of a CTA alone on its SM

int block_of(int format) { return format == MX_FP4_E4M3 ? 16 : 32; }

mx_status check_format(int format, const float *tensor_scale, const char *name)
{
    if (format != MX_FP4_E8M0 && format != MX_FP4_E4M3)
        return fail(MX_ERR_INVALID_ARG, "%s: format %d is not MX_FP4_E8M0 or MX_FP4_E4M3", name, format);
    if (tensor_scale && format != MX_FP4_E4M3)
        return fail(MX_ERR_INVALID_ARG, "%s: a tensor_scale belongs to MX_FP4_E4M3", name);
    if (!aligned(tensor_scale, 4))
        return fail(MX_ERR_ALIGNMENT, "%s: tensor_scale must be 4-byte aligned", name);
    return MX_OK;
}

mx_status check_sizes(int rows, int cols, int count, const char *name)
{
    if (rows < 1 || cols < 1 || rows > kMaxCols || cols > kMaxCols)
        return fail(MX_ERR_UNSUPPORTED, "%s: shape [%d, %d] must be within [1, %d]", name, rows, cols, kMaxCols);
    if (count < 1 || count > kMaxExperts)
        return fail(MX_ERR_UNSUPPORTED, "%s: %d matrices, at most %d are supported", name, count, kMaxExperts);
    return MX_OK;
}

mx_status check_pitch(int64_t ld, int cols, const char *name)
{
    if (ld < (cols + 1) / 2)
        return fail(MX_ERR_INVALID_ARG, "%s: row pitch %lld is below %d bytes", name, (long long)ld, (cols + 1) / 2);
    if (ld > 4 * (int64_t)kMaxCols)
        return fail(MX_ERR_UNSUPPORTED, "%s: row pitch %lld is above %d", name, (long long)ld, 4 * kMaxCols);
    return MX_OK;
}

mx_status check_matrix(const mx_fp4_matrix *m, const char *name)
{
    mx_status st;
    if (!m)
        return fail(MX_ERR_INVALID_ARG, "%s is NULL", name);
    if (!m->q || !m->scales)
        return fail(MX_ERR_INVALID_ARG, "%s has a NULL pointer", name);
    if ((st = check_format(m->format, m->tensor_scale, name)) != MX_OK ||
        (st = check_sizes(m->rows, m->cols, m->count, name)) != MX_OK || (st = check_pitch(m->ld, m->cols, name)) != MX_OK)
        return st;
    if (!aligned(m->q, 16) || m->ld % 16 || !aligned(m->scales, 16))
        return fail(MX_ERR_ALIGNMENT, "%s: addresses and the row pitch must be multiples of 16 bytes", name);
    return MX_OK;
}

mx_status check_rows(const mx_fp4_rows *r, const char *name, bool operand)
{
    mx_status st;
    if (!r)
        return fail(MX_ERR_INVALID_ARG, "%s is NULL", name);
    if (r->rows < 0 || r->rows > kMaxRows)
        return fail(MX_ERR_INVALID_ARG, "%s: %d rows must be within [0, %d]", name, r->rows, kMaxRows);
    if (r->cols < 1 || r->cols > kMaxCols)
        return fail(MX_ERR_UNSUPPORTED, "%s: %d columns must be within [1, %d]", name, r->cols, kMaxCols);
    if ((st = check_format(r->format, r->tensor_scale, name)) != MX_OK || (st = check_pitch(r->ld, r->cols, name)) != MX_OK)
        return st;
    if (r->rows == 0)
        return MX_OK;
    if (!r->q || !r->scales)
        return fail(MX_ERR_INVALID_ARG, "%s has a NULL pointer", name);
    if (operand && (!aligned(r->q, 16) || r->ld % 16))
        return fail(MX_ERR_ALIGNMENT, "%s: address and row pitch must be multiples of 16 bytes", name);
    if (!aligned(r->scales, 16))
        return fail(MX_ERR_ALIGNMENT, "%s: scales must be 16-byte aligned", name);
    return MX_OK;
}

// One row by mx_fp4_gemv.cu, while its CTAs' rounds over the SMs have few steps of 1024 columns: 2112 x 2816 (one round
// of three) 3.1 us, by the tensor cores 5.1; 2112 x 4096 3.8, 5.3; 3328 x 2816 (two of three) 4.4, 5.2; 4096 x 4096 (two of
// four) 5.5, 5.6; 704 x 8192 (one of eight) 5.4, 5.4; 14336 x 4096 14.5, 6.8.
bool one_row(int rows, const int32_t *offsets, const mx_fp4_matrix &w)
{
    const int64_t ctas = (w.rows + 127) / 128 * 8, rounds = (ctas + num_sms() - 1) / num_sms();
    return rows == 1 && !offsets && rounds * ((w.cols + 1023) / 1024) <= 6;
}

mx_status product(const mx_fp4_rows *x, const int32_t *offsets, const mx_fp4_matrix *w, void *out, int64_t ldo,
                  int out_dtype, void *stream, void *ws, size_t ws_bytes)
{
    mx_status st;
    if ((st = check_rows(x, "x", true)) != MX_OK || (st = check_matrix(w, "w")) != MX_OK ||
        (st = check_dtype(out_dtype, "out_dtype")) != MX_OK)
        return st;
    if (x->cols != w->cols || x->format != w->format)
        return fail(MX_ERR_INVALID_ARG, "x has %d columns in format %d, w has %d in format %d", x->cols, x->format, w->cols,
                    w->format);
    if (ldo < w->rows)
        return fail(MX_ERR_INVALID_ARG, "output row pitch %lld is below its %d columns", (long long)ldo, w->rows);
    if (ldo > ((int64_t)1 << 31))
        return fail(MX_ERR_UNSUPPORTED, "output row pitch %lld is too large", (long long)ldo);
    if (x->rows == 0)
        return MX_OK;
    if (!out)
        return fail(MX_ERR_INVALID_ARG, "out is NULL");
    if (!aligned(out, dtype_bytes(out_dtype)))
        return fail(MX_ERR_ALIGNMENT, "out is misaligned");
    if ((st = check_ws(ws, ws_bytes, kErrBytes)) != MX_OK)
        return st;
    const int block = block_of(w->format), FT = (w->rows + 127) / 128, KB = stages_of(w->cols);
    if (one_row(x->rows, offsets, *w)) {
        GemvArgs v{};
        v.K = w->cols;
        v.N = w->rows;
        v.q = static_cast<const uint8_t *>(x->q);
        v.sx = static_cast<const uint8_t *>(x->scales);
        v.w = static_cast<const uint8_t *>(w->q);
        v.sw = static_cast<const uint8_t *>(w->scales);
        v.ldw = w->ld;
        v.tx = x->tensor_scale;
        v.tw = w->tensor_scale;
        v.out = out;
        v.out_bf16 = out_dtype == MX_BF16;
        const cudaError_t e = launch_gemv(block, v, static_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? MX_OK : cuda_fail(e, "FP4 product");
    }
    const Choice c = choose(x->rows, offsets != nullptr, w->count, FT, KB, num_sms());
    GemmArgs g{};
    g.rows = x->rows;
    g.K = w->cols;
    g.N = w->rows;
    g.E = w->count;
    g.offsets = offsets;
    g.sx = static_cast<const uint8_t *>(x->scales);
    g.sw = static_cast<const uint8_t *>(w->scales);
    g.tx = x->tensor_scale;
    g.tw = w->tensor_scale;
    g.out = out;
    g.ldo = ldo;
    g.out_bf16 = out_dtype == MX_BF16;
    g.out_vec = vec16(out, ldo, g.out_bf16);
    g.err = static_cast<unsigned *>(ws);
    g.cl = c.cl;
    // (a CTA of several tiles loads on into the next ones: 4096 rows of 128 matrices 2816 x 704, three stages a tile, 36 us
    // with a ring of three, 30 with all that fit)
    g.stages = c.several ? 12 : std::min(12, std::max(2, KB));
    while (g.stages > 2 && gemm_smem(block, c.nt, g.stages) > (size_t)kSmem)
        --g.stages;
    const uint64_t bytes = ((uint64_t)w->cols + 1) / 2;
    cudaError_t e = tma_map_bytes(&g.wm, w->q, TmaBytes{bytes, (uint64_t)w->rows, (uint64_t)w->count, (uint64_t)w->ld, 128});
    if (e == cudaSuccess)
        e = tma_map_bytes(&g.xm, x->q, TmaBytes{bytes, (uint64_t)x->rows, 0, (uint64_t)x->ld, (uint32_t)box_rows(c.nt)});
    if (e != cudaSuccess)
        return cuda_fail(e, "tensor map of an FP4 operand");
    e = launch_gemm(block, c.nt, g, c.grid, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MX_OK : cuda_fail(e, "FP4 product");
}

}  // namespace

extern "C" mx_status mx_fp4_quantize(const void *x, int64_t ldx, int dtype, const mx_fp4_rows *out, void *stream)
{
    mx_status st;
    if ((st = check_dtype(dtype, "dtype")) != MX_OK || (st = check_rows(out, "out", false)) != MX_OK)
        return st;
    if (ldx < out->cols)
        return fail(MX_ERR_INVALID_ARG, "x: row pitch %lld is below its %d columns", (long long)ldx, out->cols);
    if (ldx > ((int64_t)1 << 31))
        return fail(MX_ERR_UNSUPPORTED, "x: row pitch %lld is too large", (long long)ldx);
    if (out->rows == 0)
        return MX_OK;
    if (!x)
        return fail(MX_ERR_INVALID_ARG, "x is NULL");
    if (!aligned(x, dtype_bytes(dtype)))
        return fail(MX_ERR_ALIGNMENT, "x is misaligned");
    QuantArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.rows = out->rows;
    a.cols = out->cols;
    a.bf16 = dtype == MX_BF16;
    a.vx = vec16(x, ldx, a.bf16);
    a.vq = aligned(out->q, 8) && out->ld % 8 == 0;
    a.q = static_cast<uint8_t *>(out->q);
    a.scales = static_cast<uint8_t *>(out->scales);
    a.ldq = out->ld;
    a.tensor_scale = out->tensor_scale;
    const cudaError_t e = launch_quantize(block_of(out->format), a, num_sms(), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MX_OK : cuda_fail(e, "FP4 quantisation");
}

extern "C" size_t mx_fp4_pack_bytes(int rows, int cols, int count, int format)
{
    if (check_format(format, nullptr, "scales") != MX_OK || check_sizes(rows, cols, count, "scales") != MX_OK)
        return 0;
    return (size_t)count * ((rows + 127) / 128) * stages_of(cols) * atoms_of(block_of(format)) * 512;
}

extern "C" mx_status mx_fp4_pack_scales(const void *scales, int64_t ld, int rows, int cols, int count, int format, void *out,
                                        void *stream)
{
    mx_status st;
    if ((st = check_format(format, nullptr, "scales")) != MX_OK || (st = check_sizes(rows, cols, count, "scales")) != MX_OK)
        return st;
    const int block = block_of(format), nb = (cols + block - 1) / block;
    if (ld < nb)
        return fail(MX_ERR_INVALID_ARG, "scales: row pitch %lld is below %d blocks", (long long)ld, nb);
    if (ld > 4 * (int64_t)kMaxCols)
        return fail(MX_ERR_UNSUPPORTED, "scales: row pitch %lld is above %d", (long long)ld, 4 * kMaxCols);
    if (!scales || !out)
        return fail(MX_ERR_INVALID_ARG, "scales and out must not be NULL");
    if (!aligned(out, 16))
        return fail(MX_ERR_ALIGNMENT, "out must be 16-byte aligned");
    PackArgs a{static_cast<const uint8_t *>(scales), ld, rows, nb, count, block, static_cast<uint8_t *>(out)};
    const cudaError_t e = launch_pack(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MX_OK : cuda_fail(e, "FP4 scales");
}

extern "C" mx_status mx_fp4_matmul(const mx_fp4_rows *x, const mx_fp4_matrix *w, void *out, int64_t ldo, int out_dtype,
                                   void *stream, void *ws, size_t ws_bytes)
{
    if (w && w->count != 1)
        return fail(MX_ERR_INVALID_ARG, "w holds %d matrices, one is needed", w->count);
    return product(x, nullptr, w, out, ldo, out_dtype, stream, ws, ws_bytes);
}

extern "C" mx_status mx_fp4_grouped_matmul(const mx_fp4_rows *x, const int32_t *offsets, const mx_fp4_matrix *w, void *out,
                                           int64_t ldo, int out_dtype, void *stream, void *ws, size_t ws_bytes)
{
    if (!offsets)
        return fail(MX_ERR_INVALID_ARG, "offsets is NULL");
    if (!aligned(offsets, 4))
        return fail(MX_ERR_ALIGNMENT, "offsets must be 4-byte aligned");
    return product(x, offsets, w, out, ldo, out_dtype, stream, ws, ws_bytes);
}

extern "C" size_t mx_fp4_matmul_workspace_bytes(const mx_fp4_matrix *w, int rows)
{
    if (check_matrix(w, "w") != MX_OK)
        return 0;
    if (rows < 0) {
        fail(MX_ERR_INVALID_ARG, "%d rows", rows);
        return 0;
    }
    return kErrBytes;
}
