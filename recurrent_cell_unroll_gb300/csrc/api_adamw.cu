// Host side of the AdamW step and of the 8-bit optimizer states of include/rcu.h:
// argument checks and the launches (adamw.cu).
#include <cmath>

#include "api_seq.h"
#include "ssm.h"

using namespace rcu;
using namespace rcu_api;
using namespace rcu_seq_api;

namespace {

int check_tensor(const char *fn, int64_t k, const rcu_adamw_tensor &t) {
  if (t.n < 0) return fail(RCU_ERR_INVALID, "%s: tensor %lld has a negative size", fn, (long long)k);
  if (t.n == 0) return RCU_OK;
  if (!t.p || !t.g || !t.m || !t.v)
    return fail(RCU_ERR_INVALID, "%s: p, g, m or v of tensor %lld is NULL", fn, (long long)k);
  if (!dtype_ok(t.p_type) || !dtype_ok(t.g_type))
    return fail(RCU_ERR_INVALID, "%s: types of tensor %lld must be RCU_F32 or RCU_BF16", fn,
                (long long)k);
  if ((t.m_exp != nullptr) != (t.v_exp != nullptr))
    return fail(RCU_ERR_INVALID, "%s: tensor %lld has exponents for one of its states only", fn,
                (long long)k);
  if (t.copy && t.p_type != RCU_F32)
    return fail(RCU_ERR_INVALID, "%s: tensor %lld has a copy of a bf16 parameter", fn, (long long)k);
  if (t.n > (int64_t)1 << (t.m_exp ? 32 : 40))
    return fail(RCU_ERR_UNSUPPORTED, "%s: tensor %lld is too large", fn, (long long)k);
  return RCU_OK;
}

int check_state8(const char *fn, rcu_seq *h, int64_t n, const void *x, const void *codes,
                 const void *exps) {
  const int rc = check_handle(fn, h);
  if (rc != RCU_OK) return rc;
  if (n < 0) return fail(RCU_ERR_INVALID, "%s: n must be >= 0", fn);
  if (n > (int64_t)1 << 40) return fail(RCU_ERR_UNSUPPORTED, "%s: n above 2^40", fn);
  if (n && (!x || !codes || !exps)) return fail(RCU_ERR_INVALID, "%s: NULL values, codes or exps", fn);
  return RCU_OK;
}

}  // namespace

extern "C" int rcu_adamw_step(rcu_seq *h, int64_t count, const rcu_adamw_tensor *tensors, double lr,
                              double beta1, double beta2, double eps, double weight_decay,
                              int64_t step, int64_t seed, const float *scale,
                              const int32_t *step_dev, const float *lr_dev, void *stream) {
  const int rc = check_handle(__func__, h);
  if (rc != RCU_OK) return rc;
  if (count < 0 || (count && !tensors))
    return fail(RCU_ERR_INVALID, "rcu_adamw_step: no list of tensors");
  if (count > 1 << 24) return fail(RCU_ERR_UNSUPPORTED, "rcu_adamw_step: more than 2^24 tensors");
  if (!(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1))
    return fail(RCU_ERR_INVALID, "rcu_adamw_step: betas must be in [0, 1)");
  if (!(eps >= 0) || !std::isfinite((float)eps) || !std::isfinite(lr) || !std::isfinite(weight_decay))
    return fail(RCU_ERR_INVALID, "rcu_adamw_step: eps must be >= 0, and lr, eps, weight_decay finite");
  if (!step_dev && step < 1) return fail(RCU_ERR_INVALID, "rcu_adamw_step: step must be >= 1");
  for (int64_t k = 0; k < count; ++k) {
    const int tc = check_tensor(__func__, k, tensors[k]);
    if (tc != RCU_OK) return tc;
  }
  cudaStream_t s = (cudaStream_t)stream;
  h->launches = 0;
  const AdamWStep p{lr, beta1, beta2, eps, weight_decay, step, (uint32_t)seed, scale, step_dev, lr_dev};
  begin(h, "adamw_step", s);
  CU(launch_adamw(p, count, tensors, h->nsm, !h->force_path, s, &h->launches));
  h->prof_end(s);
  return RCU_OK;
}

extern "C" int rcu_state8_pack(rcu_seq *h, int is_signed, int64_t n, const float *x, int8_t *codes,
                               int8_t *exps, void *stream) {
  const int rc = check_state8(__func__, h, n, x, codes, exps);
  if (rc != RCU_OK) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  h->launches = 0;
  if (n == 0) return RCU_OK;
  begin(h, "state8_pack", s);
  CU(launch_state8_pack(is_signed, n, x, codes, exps, h->nsm, !h->force_path, s, &h->launches));
  h->prof_end(s);
  return RCU_OK;
}

extern "C" int rcu_state8_unpack(rcu_seq *h, int is_signed, int64_t n, const int8_t *codes,
                                 const int8_t *exps, float *y, void *stream) {
  const int rc = check_state8(__func__, h, n, y, codes, exps);
  if (rc != RCU_OK) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  h->launches = 0;
  if (n == 0) return RCU_OK;
  begin(h, "state8_unpack", s);
  CU(launch_state8_unpack(is_signed, n, codes, exps, y, h->nsm, !h->force_path, s, &h->launches));
  h->prof_end(s);
  return RCU_OK;
}
