// The experts' gated feed-forward on fp16 values.
#include "ffn_launch.hpp"

namespace embtab {

EMBTAB_FFN_TYPE(f16_t)

}  // namespace embtab
