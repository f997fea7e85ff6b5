// The router's projection alone (moe_router_logits): the kernels of route.cu with an epilogue
// that stores each token's logits instead of choosing experts, so the logits are the bits that
// moe_route selects by.  A translation unit of its own: the two compile side by side, and the
// routing kernels' code stays as it is without this variant.
#define MOE_ROUTER_LOGITS
#include "route.cu"
