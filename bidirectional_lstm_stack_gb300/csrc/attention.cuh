// What the files of linear attention share: a call's arguments and the entry
// points' way to the kernels.
#pragma once

#include "lstm_layers.h"
#include "ops.cuh"

namespace lstm {

// Rows of heads: element (t, h, c) at t * stride + h * head_stride + c.
struct HeadRows {
    const void *at;
    long long stride, head_stride;
    int share;  // heads of the call that one head of these rows serves

    template <typename T>
    __device__ __forceinline__ const T *row(long long t, int head) const
    {
        return static_cast<const T *>(at) + t * stride + (head / share) * head_stride;
    }
};

struct AttentionArgs {
    HeadRows q, k, v;
    const float *decay;
    long long decay_stride;  // 0: the same for every token
    float scale;
    int heads, keys, values;
    float *state;
    Sequences seq;
    Slots slots;
    void *y;
    long long y_stride;

    template <typename T>
    __device__ __forceinline__ T *out(long long t, int head) const
    {
        return static_cast<T *>(y) + t * y_stride + static_cast<long long>(head) * values;
    }
    __device__ __forceinline__ long long cells() const
    {
        return static_cast<long long>(keys) * values;
    }
    // The state of a slot's head.
    __device__ __forceinline__ float *state_of(int slot, int head) const
    {
        return state + (static_cast<long long>(slot) * heads + head) * cells();
    }
};

// How prompts are cut into spans.  Spans are numbered as tile_owner() numbers tiles, so a
// sequence's follow each other.
struct Spans {
    int tokens = 0;  // of a span; 0: sequences are whole
    int units = 0;   // numbers
    float *states = nullptr;  // [units][heads][keys][values]: what each span starts from
    float *left = nullptr;    // [units][heads]: the product of its decays

    // of a sequence; one of no rows has one span too, for its state
    __device__ __forceinline__ int count(int rows) const
    {
        return rows > tokens ? (rows - 1) / tokens + 1 : 1;
    }
    __device__ __forceinline__ float *state_of(const AttentionArgs &p, int unit, int head) const
    {
        return states + (static_cast<long long>(unit) * p.heads + head) * p.cells();
    }
    __device__ __forceinline__ float *left_of(const AttentionArgs &p, int unit, int head) const
    {
        return left + static_cast<long long>(unit) * p.heads + head;
    }
};

int launch_attention_f32(const AttentionArgs &p, const Spans &spans, cudaStream_t stream);
int launch_attention_bf16(const AttentionArgs &p, const Spans &spans, cudaStream_t stream);
int launch_attention_f16(const AttentionArgs &p, const Spans &spans, cudaStream_t stream);
int launch_attention_join(const AttentionArgs &p, const Spans &spans, cudaStream_t stream);
int launch_attention_step(const AttentionArgs &p, int dtype, cudaStream_t stream);

}  // namespace lstm
