// Products of the gated block's backward pass, bf16 operands.
#include "prod_api.hpp"
#include "prod_launch.hpp"

template <>
hipError_t tg::launch_plain<1, 0>(const ProdArgs &p, const PlainEpi<0> &e, hipStream_t s) {
    return launch_prod_aligned<1>(p, e, s);
}
template <>
hipError_t tg::launch_plain<1, 1>(const ProdArgs &p, const PlainEpi<1> &e, hipStream_t s) {
    return launch_prod_aligned<1>(p, e, s);
}
