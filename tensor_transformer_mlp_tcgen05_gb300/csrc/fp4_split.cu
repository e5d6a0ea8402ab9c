// The product of few rows with a packed A (fp4_split.cuh).
#include "fp4_split.cuh"

namespace tpmlp {
namespace fp4 {
namespace {

using namespace split;

// Columns of the MMA, and with them A's share of a stage, by A's rows (128 columns
// for 8 rows: 8 x 5120 x 20480 in L2 9.7 us, not 7.8; for 64: 11.7, not 10.7).
template <int FORMAT, int EPI>
cudaError_t launch_epilogue(const ProductArgs& args, int sms, cudaStream_t s) {
  if (args.M <= 16) return launch_tokens<FORMAT, EPI, 16, PACKED>(args, sms, s);
  if (args.M <= 32) return launch_tokens<FORMAT, EPI, 32, PACKED>(args, sms, s);
  if (args.M <= 64) return launch_tokens<FORMAT, EPI, 64, PACKED>(args, sms, s);
  return launch_tokens<FORMAT, EPI, 128, PACKED>(args, sms, s);
}

template <int FORMAT>
cudaError_t launch_format(const ProductArgs& args, int sms, cudaStream_t s) {
  switch (args.epilogue) {
    case OUT_BF16: return launch_epilogue<FORMAT, OUT_BF16>(args, sms, s);
    case OUT_FP32: return launch_epilogue<FORMAT, OUT_FP32>(args, sms, s);
    default: return launch_epilogue<FORMAT, OUT_GELU_FP4>(args, sms, s);
  }
}

}  // namespace

cudaError_t launch_product_split(int format, const ProductArgs& args, int sms,
                                 cudaStream_t s) {
  if (args.x != nullptr) return launch_product_plain(format, args, sms, s);
  return format == TPFP4_NV ? launch_format<TPFP4_NV>(args, sms, s)
                            : launch_format<TPFP4_MX>(args, sms, s);
}

}  // namespace fp4
}  // namespace tpmlp
