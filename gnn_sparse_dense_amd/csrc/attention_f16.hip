// Attention within segments, rows of f16.
#include "attention_impl.h"

namespace gspmm {

ATTENTION_OF(_Float16);

}  // namespace gspmm
