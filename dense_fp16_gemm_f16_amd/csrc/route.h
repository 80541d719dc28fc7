// Routing to experts and the way back from them (host interface of route.hip and
// combine.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

namespace gemm_f16 {

constexpr int kRouteExperts = 2048, kRouteFan = 32, kRouteGroups = 64;

struct RouteParams {
    const void *logits;    // [tokens, experts], fp16 or fp32
    const float *bias;     // [experts] or null
    int32_t *ids;          // [tokens, fan]
    float *gates;          // [tokens, fan]
    const float *dgates;   // gradient: [tokens, fan]
    void *dlogits;         // gradient: [tokens, experts], of the logits' type
    int64_t tokens, first;  // first: tokens that earlier launches hold
    int32_t experts, fan, f32, sigmoid, groups, top_groups, group_top, renormalize;
    int32_t vec, bias_vec; // rows, the bias in whole aligned chunks of 4
    float scale;
};
hipError_t launch_route(const RouteParams &p, hipStream_t s);
hipError_t launch_route_grad(const RouteParams &p, hipStream_t s);

struct CombineParams {
    const void *rows;        // [tokens fan, n], fp16 or fp32
    const int32_t *inverse;  // [tokens, fan]
    const int32_t *last;     // places from *last on belong to no group
    const float *gates;      // [tokens, fan], or null: ones
    const void *residual;    // [tokens, n] of y's type, or null; y itself, or apart from it
    void *y;                 // [tokens, n], fp16 or fp32; gradient: dy, read
    void *drows;             // gradient: [tokens fan, n], fp16 or fp32, or null
    float *dgates;           // gradient: [tokens, fan], or null
    int64_t tokens, places, first;  // places: tokens fan; first: tokens that earlier launches hold
    int32_t fan, n, rows_f32, y_f32, drows_f32;
};
hipError_t launch_combine(const CombineParams &p, hipStream_t s);
hipError_t launch_combine_grad(const CombineParams &p, hipStream_t s);

}  // namespace gemm_f16
