// Gated block, fp16.
#include "prod_api.hpp"
#include "prod_launch.hpp"

template <>
hipError_t tg::launch_glu<2>(const ProdArgs &p, const GluEpi<2> &e, hipStream_t s) {
    return launch_prod<2, true>(p, e, s);
}
