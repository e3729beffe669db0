// C ABI of the products grouped by expert (vq_experts_*): argument checks, the handle, and the
// choice of the kernel.
#include <new>

#include "api_util.h"
#include "experts.cuh"

namespace vq {
cudaError_t launch_experts_gemv(const ExpertsArgs& a, int num_sms, cudaStream_t s);
cudaError_t launch_experts_tc(const ExpertsArgs& a, void* xs, int Tmax, int num_sms, cudaStream_t s);
}  // namespace vq

using namespace vq;

struct vq_experts_s {
  vq_experts_desc d;  // first, as in vq_linear_s
  DeviceInfo dev;
  int path;
  uint32_t* err;  // device word, set by bounded waits that gave up
  void* xs;       // [max_M][K]: x in row order, for the tensor-core kernel (desc.gather == 1)
};

namespace {

struct ExpertsPlan {
  int path;  // VQ_PATH_GEMV or VQ_PATH_TC
  int Tmax;  // rows of a tile
};

// The kernel, from T, E and the layer (the row counts themselves are on the device): `busy`
// experts can have rows, `avg` each.  The tensor-core kernel decodes 2.4 T weights a second for up to
// 256 rows, once its tiles of 256 rows of W fill the SMs; the warp-MMA kernel as many for up to 8, and
// again for every 16 rows that an expert has, in tiles of 16 rows of W that fill the SMs sooner, and
// it starts faster.  Measured, us, warp-MMA / tensor-core: 64 experts x 1 row (2048 x 1024, 512
// tiles) 54 / 56, x 8 (up to 18) 74 / 56, x 32 179 / 57; 8 x 1 (2048 x 2048 gated, 64 tiles) 18.0 /
// 20.7, x 16 21.3 / 20.8; 8 x 2 (1024 x 576, 32 tiles) 8.5 / 13.0; 2 x 1 (2048 x 2048 gated, 16
// tiles) 9.4 / 19.6; 16-bit indices, 16 x 12 (1536 x 576, 96 tiles) 19.4 / 21.8, x 25 27.5 / 22.7.
// The formats share the thresholds, and the shape counts only through the SMs.  Over 6300 random calls (2 to
// 128 experts of up to 4096 x 4096, 1 to 100 rows on average) the choice takes 1.09 times as long as the
// faster kernel on 12-bit formats, 1.22 on 16-bit ones and 1.14 on the ladder (geometric means); at
// worst 2.9, 4.8 and 6.6 times, where fewer than 74 tiles (3 experts of 128 x 4096) leave most pairs of the
// tensor-core kernel without one.  The average says nothing of the spread: 128 rows that all go to
// one of 64 experts run on the warp-MMA kernel, which decodes that expert's weights eight times.
ExpertsPlan plan_experts(const vq_experts_desc& d, int T, int forced, int num_sms) {
  const int busy = T < d.E ? T : d.E;
  const int avg = (T + busy - 1) / busy;
  const int64_t tiles = (int64_t)busy * ((d.layer.N + 255) / 256);
  ExpertsPlan p{};
  p.path = forced != VQ_PATH_AUTO ? forced : avg <= 2 || (avg <= 14 && tiles < num_sms) ? VQ_PATH_GEMV : VQ_PATH_TC;
  // Tiles of up to 128 rows of x have a second accumulator; above, larger tiles save decodes.
  p.Tmax = p.path == VQ_PATH_GEMV ? 16 : avg <= 64 ? 128 : 256;
  return p;
}

vq_status validate_experts(const vq_experts_desc* d) {
  if (d == nullptr) return fail(VQ_ERR_INVALID_ARG, "desc is NULL");
  vq_status st = validate_desc(&d->layer);
  if (st) return st;
  if (d->E < 1) return fail(VQ_ERR_INVALID_ARG, "E=%d must be positive", d->E);
  if (d->E > kMaxExperts) return fail(VQ_ERR_UNSUPPORTED, "E=%d: at most %d experts", d->E, kMaxExperts);
  if (d->shared_codebooks != 0 && d->shared_codebooks != 1)
    return fail(VQ_ERR_INVALID_ARG, "shared_codebooks=%d must be 0 or 1", d->shared_codebooks);
  if (d->glu != 0 && d->glu != 1) return fail(VQ_ERR_INVALID_ARG, "glu=%d must be 0 or 1", d->glu);
  if (d->gather != 0 && d->gather != 1) return fail(VQ_ERR_INVALID_ARG, "gather=%d must be 0 or 1", d->gather);
  if (d->act < VQ_ACT_NONE || d->act > VQ_ACT_GELU_TANH)
    return fail(VQ_ERR_INVALID_ARG, "act=%d is not a VQ_ACT_*", d->act);
  if (d->layer.rht || d->layer.corr)
    return fail(VQ_ERR_UNSUPPORTED, "rht and corr must be 0: rotate x with vq_rht_apply; experts carry no correction");
  if (d->layer.N % (d->glu ? 16 : 8) != 0)
    return fail(VQ_ERR_UNSUPPORTED, "N=%d must be a multiple of %d", d->layer.N, d->glu ? 16 : 8);
  if ((int64_t)d->layer.N * (d->layer.K / 8) > INT32_MAX)
    return fail(VQ_ERR_UNSUPPORTED, "N=%d x K=%d: an expert may have at most 2^31 - 1 groups", d->layer.N, d->layer.K);
  // the tiles of a call are counted in 32 bits: at most 8 outputs by 16 rows each
  const int64_t rt = (d->layer.N / (d->glu ? 2 : 1) + 7) / 8;
  if (rt * ((int64_t)d->layer.max_M / 16 + d->E) > INT32_MAX)
    return fail(VQ_ERR_UNSUPPORTED, "N=%d, max_M=%d and E=%d give too many tiles", d->layer.N, d->layer.max_M, d->E);
  return VQ_OK;
}

}  // namespace

VQ_API vq_status vq_experts_create(const vq_experts_desc* desc, vq_experts_t* out) {
  if (out == nullptr) return fail(VQ_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  vq_status st = validate_experts(desc);
  if (st) return st;
  DeviceInfo dev{};
  if ((st = query_device(&dev))) return st;
  if ((st = refuse_alloc())) return st;
  vq_experts_s* h = new (std::nothrow) vq_experts_s{};
  if (!h) return fail(VQ_ERR_NOMEM, "host allocation of the handle failed");
  h->d = *desc;
  h->dev = dev;
  h->path = VQ_PATH_AUTO;
  cudaError_t e = cudaMalloc(&h->err, sizeof(uint32_t));
  const size_t xs_bytes = desc->gather ? (size_t)desc->layer.max_M * desc->layer.K * 2 : 0;
  if (e == cudaSuccess && xs_bytes) e = cudaMalloc(&h->xs, xs_bytes);
  if (e == cudaSuccess) e = cudaMemset(h->err, 0, sizeof(uint32_t));
  if (e == cudaSuccess) e = cudaDeviceSynchronize();  // the zeroing is complete before any forward
  if (e != cudaSuccess) {
    cudaFree(h->err);
    cudaFree(h->xs);
    delete h;
    cudaGetLastError();
    return fail(VQ_ERR_NOMEM, "cudaMalloc of the error word and %zu bytes for x failed: %s", xs_bytes, cudaGetErrorString(e));
  }
  *out = h;
  return VQ_OK;
}

VQ_API vq_status vq_experts_destroy(vq_experts_t h) {
  if (h == nullptr) return VQ_OK;
  cudaError_t e = free_on_device(h->dev.device, h->err, h->xs);
  delete h;
  return e == cudaSuccess ? VQ_OK : cuda_fail(e, "vq_experts_destroy");
}

VQ_API vq_status vq_experts_set_path(vq_experts_t h, int32_t path) {
  if (h == nullptr) return fail(VQ_ERR_INVALID_ARG, "handle is NULL");
  if (path != VQ_PATH_AUTO && path != VQ_PATH_GEMV && path != VQ_PATH_TC)
    return fail(VQ_ERR_INVALID_ARG, "path=%d is not VQ_PATH_AUTO, VQ_PATH_GEMV or VQ_PATH_TC", path);
  h->path = path;
  return VQ_OK;
}

VQ_API vq_status vq_experts_plan(vq_experts_t h, int32_t T, vq_plan_info* out) {
  if (h == nullptr || out == nullptr) return fail(VQ_ERR_INVALID_ARG, "handle or out is NULL");
  if (T < 1 || T > h->d.layer.max_M) return fail(VQ_ERR_INVALID_ARG, "T=%d outside [1, max_M=%d]", T, h->d.layer.max_M);
  const ExpertsPlan p = plan_experts(h->d, T, h->path, h->dev.num_sms);
  out->path = p.path;
  out->launches = p.path == VQ_PATH_TC && h->d.gather ? 2 : 1;
  out->ctas = p.path == VQ_PATH_TC ? h->dev.num_sms / 2 * 2 : h->dev.num_sms;
  out->splits = 1;
  return VQ_OK;
}

VQ_API vq_status vq_experts_forward(vq_experts_t h, const void* x, int32_t x_rows, const int32_t* rows,
                                    const int32_t* offsets, const vq_planes* planes, const vq_codebooks* codebooks,
                                    const void* scales, const void* bias, void* y, int32_t T, void* stream) {
  if (h == nullptr) return fail(VQ_ERR_INVALID_ARG, "handle is NULL");
  const vq_linear_desc& d = h->d.layer;
  if (T < 0 || T > d.max_M) return fail(VQ_ERR_INVALID_ARG, "T=%d outside [0, max_M=%d]", T, d.max_M);
  if (T == 0) return VQ_OK;
  if (x_rows < 1 || (rows == nullptr && x_rows < T))
    return fail(VQ_ERR_INVALID_ARG, "x_rows=%d: need at least %d", x_rows, rows ? 1 : T);
  if (rows && !h->d.gather) return fail(VQ_ERR_INVALID_ARG, "rows given, but the handle was created with gather = 0");
  vq_status st;
  if ((st = check_ptr(x, "x")) || (st = check_ptr(y, "y")) || (st = check_ptr(offsets, "offsets")) ||
      (st = validate_planes(d, planes)) || (st = validate_codebooks(d, codebooks, scales)))
    return st;
  if ((rows && (st = check_ptr(rows, "rows"))) || (bias && (st = check_ptr(bias, "bias")))) return st;
  const int Nout = h->d.glu ? d.N / 2 : d.N;
  const size_t yb = (size_t)T * Nout * 2;
  if (overlaps(x, (size_t)x_rows * d.K * 2, y, yb)) return fail(VQ_ERR_INVALID_ARG, "y overlaps x");
  if (overlaps(offsets, sizeof(int32_t) * (h->d.E + 1), y, yb) || (rows && overlaps(rows, sizeof(int32_t) * T, y, yb)) ||
      (bias && overlaps(bias, (size_t)h->d.E * d.N * 2, y, yb)))
    return fail(VQ_ERR_INVALID_ARG, "y overlaps offsets, rows or bias");
  if ((st = check_output(d, *planes, *codebooks, scales, h->d.E, h->d.shared_codebooks ? 1 : h->d.E, y, yb))) return st;
  if ((st = check_current_device(h->dev.device))) return st;
  ExpertsArgs a{};
  a.w = make_args(d, planes, codebooks, scales);
  a.x = static_cast<const uint16_t*>(x);
  a.y = static_cast<uint16_t*>(y);
  a.rows = rows;
  a.offsets = offsets;
  a.bias = static_cast<const uint16_t*>(bias);
  a.err = h->err;
  a.E = h->d.E;
  a.T = T;
  a.x_rows = x_rows;
  a.Nout = Nout;
  a.act = h->d.act;
  a.glu = h->d.glu;
  a.shared = h->d.shared_codebooks;
  const ExpertsPlan p = plan_experts(h->d, T, h->path, h->dev.num_sms);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = p.path == VQ_PATH_TC ? launch_experts_tc(a, h->xs, p.Tmax, h->dev.num_sms, s)
                                       : launch_experts_gemv(a, h->dev.num_sms, s);
  return e == cudaSuccess ? VQ_OK : cuda_fail(e, "vq_experts_forward launch");
}

VQ_API vq_status vq_experts_check(vq_experts_t h, void* stream) {
  if (h == nullptr) return fail(VQ_ERR_INVALID_ARG, "handle is NULL");
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
  uint32_t flag = 0;
  e = cudaMemcpy(&flag, h->err, sizeof flag, cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fail(e, "reading the error word");
  if (flag) {
    e = cudaMemset(h->err, 0, sizeof(uint32_t));
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_fail(e, "clearing the error word");
    return fail(VQ_ERR_TIMEOUT, "a bounded device wait gave up (flag 0x%x)", flag);
  }
  return VQ_OK;
}
