// Attention within segments, rows of bf16.
#include "attention_impl.h"

namespace gspmm {

ATTENTION_OF(__bf16);

}  // namespace gspmm
