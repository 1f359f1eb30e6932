// The experts' gated feed-forward on bf16 values.
#include "ffn_launch.hpp"

namespace embtab {

EMBTAB_FFN_TYPE(bf16_t)

}  // namespace embtab
