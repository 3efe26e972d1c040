// libspecdec.cu — the library's translation unit: the verifier, then the calls
// around the verify step.  They are separate files because a measurement of the
// verifier (its memory traffic, by a hash of its sources) holds until those change.
#include "specdec_api.cu"

#include "decode_api.cuh"
