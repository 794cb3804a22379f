// Products of 8-bit integers, f32 results.
#include "prod_api.hpp"
#include "prod_launch.hpp"

template <>
hipError_t tg::launch_int8<0>(const ProdArgs &p, const Int8Epi<0> &e, hipStream_t s) {
    return launch_prod<kI8, false>(p, e, s);
}
