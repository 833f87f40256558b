/*
 * The norms and the joined products linked against the stand-in for the CUDA runtime of experts_on_fake_device.c: the
 * same report for each call.  No pointer to the device is dereferenced.
 */
#define main experts_main
#include "experts_on_fake_device.c"
#undef main

int main(int argc, char **argv)
{
    char *a = (char *)0x10000, *b = (char *)0x20000, *c = (char *)0x30000, *d = (char *)0x40000, *e = (char *)0x50000;
    const void *grads[2] = {a, b};
    static const void *many[2000];
    static int64_t sizes[2000];
    static int types[2000];
    int i;
    g_major = argc > 1 ? atoi(argv[1]) : 10;
    for (i = 0; i < 2000; ++i) many[i] = a, sizes[i] = 1000;
    report("moe_expert_swiglu", moe_expert_swiglu(a, b, 0, c, d, 0, (int32_t *)e, 64, 4, 128, 128, a, b, c, d, 0, NULL, NULL));
    report("moe_expert_swiglu_backward", moe_expert_swiglu_backward(a, b, 0, c, d, 0, (int32_t *)e, a, b, 0, 64, 4, 128, 128, c, d, e,
                                                                     0, NULL, NULL));
    report("moe_rms_norm", moe_rms_norm(a, b, c, 0, 1e-6f, 10, 1024, d, e, a, b, 0, (float *)c, NULL));
    report("moe_rms_norm:most", moe_rms_norm(a, NULL, c, 0, 1e-6f, 2147483647, 16384, NULL, e, NULL, NULL, 0, NULL, NULL));
    report("moe_rms_norm_backward", moe_rms_norm_backward(a, b, c, 0, (float *)d, NULL, NULL, 100000, 1024, e, (float *)a, NULL, b,
                                                          moe_rms_norm_backward_workspace_size(100000, 1024), NULL));
    report("moe_rms_norm_backward:none", moe_rms_norm_backward(NULL, NULL, c, 0, NULL, NULL, NULL, 0, 1024, NULL, (float *)a, NULL, b, 0, NULL));
    report("moe_grad_norm", moe_grad_norm(grads, sizes, types, 2, (float *)c, d, moe_grad_norm_workspace_size(2), NULL));
    report("moe_grad_norm:none", moe_grad_norm(NULL, NULL, NULL, 0, (float *)c, d, moe_grad_norm_workspace_size(0), NULL));
    report("moe_clip_grad_norm", moe_clip_grad_norm(grads, NULL, sizes, types, 2, 1.0, (float *)c, d, moe_grad_norm_workspace_size(2), NULL));
    report("moe_clip_grad_norm:many", moe_clip_grad_norm(many, NULL, sizes, types, 2000, 1.0, (float *)c, d,
                                                         moe_grad_norm_workspace_size(2000), NULL));
    sizes[0] = 0;
    grads[0] = (char *)0x10003; /* of a tensor without elements nothing is looked at */
    report("moe_grad_norm:empty", moe_grad_norm(grads, sizes, types, 2, (float *)c, d, moe_grad_norm_workspace_size(2), NULL));
    return 0;
}
