// Products of the gated block's backward pass, fp16 operands.
#include "prod_api.hpp"
#include "prod_launch.hpp"

template <>
hipError_t tg::launch_plain<2, 0>(const ProdArgs &p, const PlainEpi<0> &e, hipStream_t s) {
    return launch_prod_aligned<2>(p, e, s);
}
template <>
hipError_t tg::launch_plain<2, 2>(const ProdArgs &p, const PlainEpi<2> &e, hipStream_t s) {
    return launch_prod_aligned<2>(p, e, s);
}
