// The library as one translation unit: the fast-weight layer, and the
// operators of the block around it on the same host services (error text,
// timing, device check).
#include "lact.hip"
#include "lact_block.hpp"
