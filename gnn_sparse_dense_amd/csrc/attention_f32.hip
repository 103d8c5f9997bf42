// Attention within segments, rows of f32.
#include "attention_impl.h"

namespace gspmm {

ATTENTION_OF(float);

}  // namespace gspmm
