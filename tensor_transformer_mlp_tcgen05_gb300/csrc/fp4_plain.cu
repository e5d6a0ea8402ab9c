// The product of up to 8 rows that it quantises itself (fp4_split.cuh).
#include "fp4_split.cuh"

namespace tpmlp {
namespace fp4 {
namespace {

using namespace split;

template <int FORMAT>
cudaError_t launch_format(const ProductArgs& args, int sms, cudaStream_t s) {
  constexpr int NT = 16;
  if (args.M > 4) {   // bf16
    switch (args.epilogue) {
      case OUT_BF16: return launch_tokens<FORMAT, OUT_BF16, NT, PLAIN_BF16_8>(args, sms, s);
      case OUT_FP32: return launch_tokens<FORMAT, OUT_FP32, NT, PLAIN_BF16_8>(args, sms, s);
      default: return launch_tokens<FORMAT, OUT_GELU_FP4, NT, PLAIN_BF16_8>(args, sms, s);
    }
  }
  if (args.epilogue == OUT_GELU_FP4)   // the MLP block's: bf16
    return launch_tokens<FORMAT, OUT_GELU_FP4, NT, PLAIN_BF16>(args, sms, s);
  if (args.epilogue == OUT_BF16)
    return args.x_bf16
               ? launch_tokens<FORMAT, OUT_BF16, NT, PLAIN_BF16>(args, sms, s)
               : launch_tokens<FORMAT, OUT_BF16, NT, PLAIN_FP32>(args, sms, s);
  return args.x_bf16
             ? launch_tokens<FORMAT, OUT_FP32, NT, PLAIN_BF16>(args, sms, s)
             : launch_tokens<FORMAT, OUT_FP32, NT, PLAIN_FP32>(args, sms, s);
}

}  // namespace

cudaError_t launch_product_plain(int format, const ProductArgs& args, int sms,
                                 cudaStream_t s) {
  return format == TPFP4_NV ? launch_format<TPFP4_NV>(args, sms, s)
                            : launch_format<TPFP4_MX>(args, sms, s);
}

}  // namespace fp4
}  // namespace tpmlp
