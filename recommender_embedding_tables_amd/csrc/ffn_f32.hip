// The experts' gated feed-forward on fp32 values.
#include "ffn_launch.hpp"

namespace embtab {

EMBTAB_FFN_TYPE(float)

}  // namespace embtab
